"""Norm and clipping of a list of gradients on the GPU against 64-bit values:
lists of none to thousands, lengths 0 to millions, every alignment, values that
fp32 cannot square, NaN and infinity, in place and into a flat buffer."""
import math

import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import layers_reference as ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F, B = zs.ZS_FP32, zs.ZS_BF16
TYPE = ref.DTYPES


def _list(seed, lengths, dtype, sigma=1.0, offset=0):
    """Tensors of the lengths, `offset` elements into allocations of their own."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [(torch.randn(n + offset, generator=g, device=DEV) * sigma).to(TYPE[dtype])[offset:]
            for n in lengths]


class Out:
    def __init__(self):
        self.ws = torch.full((zs.zs_grad_norm_workspace_bytes(),), 0xAB, dtype=torch.uint8, device=DEV)
        self.norm, self.coef = torch.full((2, 1), -3.0, device=DEV)
        self.bad = torch.full((1,), -3, dtype=torch.int32, device=DEV)
        self.sq = torch.full((1,), -3.0, dtype=torch.float64, device=DEV)

    def clip(self, tensors, dt, max_norm, outs, od, **kw):
        zs.zs_tensors_clip(tensors, dt, max_norm, outs, od, self.ws, self.norm, self.coef, self.bad, **kw)


LISTS = {
    "one": [1], "short": [7, 0, 1, 2, 255, 256, 257], "tiny model": [256000] + [256, 65536, 768] * 20,
    "chunks": [8191, 8192, 8193, 16384, 1, 3 * 8192 + 5], "many": [i % 37 for i in range(2001)],
    "large": [3_000_001, 17, 1_000_000],
}


@pytest.mark.parametrize("dt,od", [(B, B), (B, F), (F, B), (F, F)])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("name", LISTS)
def test_clip_into_a_flat_buffer(name, dt, od, offset):
    lengths = LISTS[name]
    grads = _list(len(lengths), lengths, dt, offset=offset)
    flat = torch.full((sum(lengths) + offset + 8,), 77.0, dtype=TYPE[od], device=DEV)
    outs = list(torch.split(flat[offset:offset + sum(lengths)], lengths))
    o = Out()
    sq = ref.sqnorm([t.cpu() for t in grads])
    norm = math.sqrt(sq)
    max_norm = 0.37 * norm if norm else 1.0
    zs.zs_tensors_sqnorm(grads, dt, o.ws, o.sq)
    assert abs(o.sq.item() - sq) <= ref.T_SQNORM * sq
    o.clip(grads, dt, max_norm, outs, od)
    coef = o.coef.item()
    assert o.bad.item() == 0
    # the root halves the error; the norm and the coefficient are rounded to fp32
    assert abs(o.norm.item() - norm) <= (ref.T_SQNORM / 2 + ref.EPS) * norm
    want = min(1.0, max_norm / (norm + 1e-6))
    assert abs(coef - want) <= (ref.T_SQNORM / 2 + 2 * ref.EPS) * want
    ref_flat = torch.cat([t.cpu().double() for t in grads]) * coef
    ref.close(flat[offset:offset + sum(lengths)], ref_flat,
              ref.EPS * ref_flat.abs() + ref.rounding(ref_flat, TYPE[od]), "flat")
    assert (flat[:offset] == 77.0).all() and (flat[offset + sum(lengths):] == 77.0).all()
    # in parts, as several ranks do it: the same coefficient and bits
    coef2, bad2 = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    zs.zs_clip_coefficient(o.sq, 1, max_norm, coef2, bad2)
    first = flat.clone()
    flat.fill_(77.0)
    zs.zs_tensors_scale(grads, dt, coef2, bad2, outs, od)
    assert torch.equal(coef2, o.coef) and torch.equal(first, flat)


@pytest.mark.parametrize("dt", [B, F])
def test_clip_in_place(dt):
    grads = _list(1, [1000, 3, 70001], dt)
    keep = [t.clone() for t in grads]
    handle, o = zs.Tensors(grads), Out()
    o.clip(handle, dt, 1e9, handle, dt)
    assert o.coef.item() == 1.0 and all(torch.equal(a, b) for a, b in zip(grads, keep))
    o.clip(handle, dt, 0.5, handle, dt)
    for a, b in zip(grads, keep):
        want = b.cpu().double() * o.coef.item()
        ref.close(a, want, ref.EPS * want.abs() + ref.rounding(want, TYPE[dt]), "scaled")


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", [B, F])
def test_a_norm_that_is_not_finite_changes_nothing(dt, value):
    grads = _list(2, [300, 8200, 9], dt)
    grads[1][8199] = value
    keep = [t.clone() for t in grads]
    o = Out()
    o.clip(grads, dt, 0.1, grads, dt)
    assert o.bad.item() == 1 and o.coef.item() == 1.0 and not math.isfinite(o.norm.item())
    assert all(torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) for a, b in zip(grads, keep))
    outs = [torch.full_like(t, 77.0) for t in grads]
    o.clip(grads, dt, 0.1, outs, dt)
    assert all((t == 77.0).all() for t in outs)


@pytest.mark.parametrize("sigma", [1e-38, 1e-30, 1e-22, 1e19, 1e30, 1e37])
def test_values_whose_squares_leave_fp32(sigma):
    grads = _list(3, [5000, 77], F, sigma)
    grads[0][100:4000] = 0.0
    sq = ref.sqnorm([t.cpu() for t in grads])
    o = Out()
    zs.zs_tensors_sqnorm(grads, F, o.ws, o.sq)
    assert abs(o.sq.item() - sq) <= ref.T_SQNORM * sq


def test_one_large_value_among_small_ones():
    t = torch.full((1 << 20,), 1e-3, device=DEV)
    t[12345] = 3e38
    o = Out()
    zs.zs_tensors_sqnorm([t], F, o.ws, o.sq)
    sq = ref.sqnorm([t.cpu()])
    assert abs(o.sq.item() - sq) <= ref.T_SQNORM * sq


def test_empty_lists():
    o = Out()
    o.clip([], F, 1.0, [], F)
    assert o.norm.item() == 0.0 and o.coef.item() == 1.0 and o.bad.item() == 0
    none = torch.empty(0, device=DEV)
    o = Out()
    o.clip([none, none], F, 1.0, [none, none], F)
    assert o.norm.item() == 0.0 and o.coef.item() == 1.0 and o.bad.item() == 0
    zs.zs_tensors_sqnorm([], F, o.ws, o.sq)
    assert o.sq.item() == 0.0


def test_a_tensor_past_32_bits():
    n = (1 << 32) + 5
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[-1], t[0], t[1 << 31] = 3.0, 4.0, 12.0
    o = Out()
    o.clip([t], B, 1.3, [t], B)
    assert o.norm.item() == 13.0
    want = torch.tensor([4.0, 12.0, 3.0]) * o.coef.item()
    assert torch.equal(torch.stack([t[0], t[1 << 31], t[-1]]).cpu(), want.bfloat16())


def test_the_same_tensor_twice_and_two_dtypes():
    a, b = _list(4, [4000, 500], F), _list(5, [900], B)
    o, sums = Out(), torch.zeros(2, dtype=torch.float64, device=DEV)
    zs.zs_tensors_sqnorm([a[0], a[1], a[0]], F, o.ws, sums[:1])
    zs.zs_tensors_sqnorm(b, B, o.ws, sums[1:])
    zs.zs_clip_coefficient(sums, 2, 0.5, o.coef, o.bad)
    sq = ref.sqnorm([t.cpu() for t in (a[0], a[1], a[0], b[0])])
    assert abs(sums.sum().item() - sq) <= (ref.T_SQNORM + ref.EPS) * sq
    assert abs(o.coef.item() - 0.5 / (math.sqrt(sq) + 1e-6)) <= 6 * ref.EPS * o.coef.item()
    with pytest.raises(zs.ZsError):   # as an output, in place, it would be written twice
        zs.zs_tensors_scale([a[0], a[0]], F, o.coef, None, [a[0], a[0]], F)


def test_graph_and_another_stream():
    lengths = [4096, 77, 30000]
    grads = _list(6, lengths, F)
    outs = [torch.zeros_like(t) for t in grads]
    o = Out()
    o.clip(grads, F, 1.0, outs, F)
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    o.clip(grads, F, 1.0, outs, F, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.clip(grads, F, 1.0, outs, F)
    for a, b in zip(grads, _list(7, lengths, F)):
        a.copy_(b)
    graph.replay()
    sq = ref.sqnorm([t.cpu() for t in grads])
    assert abs(o.norm.item() - math.sqrt(sq)) <= (ref.T_SQNORM / 2 + ref.EPS) * math.sqrt(sq)


def test_skip_and_coefficient_of_one():
    grads = _list(8, [5000, 33], F)
    outs = [torch.full_like(t, 77.0) for t in grads]
    coef, skip = torch.ones(1, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    zs.zs_tensors_scale(grads, F, coef, skip, outs, F)
    assert all((t == 77.0).all() for t in outs)
    skip.zero_()
    zs.zs_tensors_scale(grads, F, coef, skip, outs, F)
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    zs.zs_tensors_scale(grads, F, coef * 0.5, None, outs, F)
    assert all(torch.equal(a, b * 0.5) for a, b in zip(outs, grads))
