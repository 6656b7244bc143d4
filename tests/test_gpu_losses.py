"""The vocabulary-row losses and their gradients on the GPU against the 64-bit
reference (loss_reference.py, whose bounds these tests use)."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import loss_reference as ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: zs.ZS_BF16, torch.float32: zs.ZS_FP32}
BF16, FP32 = torch.bfloat16, torch.float32
CANARY = 777.0


def _rows(R, V, stride, dtype, lead=0, seed=0, sigma=2.5, mask=None):
    """R x V logits on the device inside a canary-filled buffer: `lead` elements
    before the first row, rows `stride` apart. Returns (buffer, view, float64)."""
    g = torch.Generator().manual_seed(seed * 7919 + V)
    buf = torch.full((lead + R * stride + 8,), CANARY, dtype=dtype)
    view = torch.as_strided(buf, (R, V), (stride, 1), lead)
    z = torch.randn(R, V, generator=g) * sigma
    hot = torch.randint(0, V, (R, 1), generator=g)
    z.scatter_(1, hot, (torch.randn(R, 1, generator=g).abs() * 4 + 4))
    view.copy_(z.to(dtype))
    if mask is not None:
        drop = torch.rand(R, V, generator=g) < 0.3
        view[drop] = -math.inf if mask == "inf" else torch.finfo(dtype).min
    dev = buf.to(DEV)
    dview = torch.as_strided(dev, (R, V), (stride, 1), lead)
    return dev, dview, view.double(), g


def _targets(R, V, g):
    t = torch.randint(0, V, (R,), generator=g)
    t[R // 2] = -100
    return t


def _f32(R):
    return torch.full((R,), CANARY, dtype=FP32, device=DEV)


def _assert_within(got, want, tol, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    # a value past the output type's range is an infinity there
    want = torch.where(want.abs() > torch.finfo(FP32).max, want * math.inf, want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~same & ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        t = tol if not torch.is_tensor(tol) else tol.expand(got.shape).flatten()[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got.flatten()[i]} for {want.flatten()[i]}, bound {t}")


def _check_logprobs(R, V, dtype, T=1.0, stride=None, lead=0, k=0, mask=None, z=None, targets=None,
                    seed=0):
    stride = stride or V
    buf, view, z64, g = _rows(R, V, stride, dtype, lead, seed, mask=mask)
    if z is not None:
        view.copy_(z.to(dtype))
        z64 = view.cpu().double()
    targets = _targets(R, V, g) if targets is None else targets
    logprob, entropy, lse = _f32(R), _f32(R), _f32(R)
    ids = torch.full((R, max(k, 1)), -7, dtype=torch.int32, device=DEV)
    tops = torch.full((R, max(k, 1)), CANARY, dtype=FP32, device=DEV)
    before = buf.clone()
    zs.zs_token_logprobs(view, CODE[dtype], R, V, stride, targets.to(DEV), T, logprob, entropy,
                         lse, k, ids if k else None, tops if k else None)
    torch.cuda.synchronize()
    assert torch.equal(buf.view(torch.uint8), before.view(torch.uint8)), "logits were written"
    o = ref.token_logprobs(z64, targets, T)
    _assert_within(lse, o["lse"], ref.tol_lse(z64, o["lse"], T), "lse")
    _assert_within(logprob, o["logprob"], ref.tol_logprob(z64, o["logprob"], T, V), "logprob")
    _assert_within(entropy, o["entropy"], ref.tol_entropy(V), "entropy")
    if k:
        want = ref.top(z64, k)
        assert torch.equal(ids.cpu().long(), want), "top ids"
        w = o["lnp"].gather(1, want)
        _assert_within(tops, w, ref.tol_logprob(z64, w, T, V), "top logprobs")
    else:
        assert bool((ids == -7).all())
    return logprob, entropy, lse, ids, tops


VOCABS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 65, 127, 129, 255, 257, 511, 1000, 1023,
          2049, 4095, 4099, 8191, 8209, 16385, 32000, 50257, 65537, 151936, 262147, 1048576]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", VOCABS)
def test_logprobs_sizes(V, dtype):
    _check_logprobs(3, V, dtype, T=0.8, k=min(V, 20))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("R,V", [(1, 50257), (2, 151936), (5, 1000), (64, 20001), (151, 4097),
                                 (153, 33000), (305, 9999), (700, 1000), (1217, 2500),
                                 (2500, 301)])
def test_logprobs_rows(R, V, dtype):
    _check_logprobs(R, V, dtype, k=5)
    _check_logprobs(R, V, dtype, T=1.7)


def test_rows_in_clusters_more_than_the_gpu_holds():
    """Rows whose table (alternatives) or whose rows in flight (loss and gradient)
    take several blocks a row although rows are many."""
    _check_logprobs(200, 262147, FP32, k=5)
    _check_distill(400, 90001, 8, BF16, T=1.5)
    _check_distill(160, 50021, 8, FP32, in_place=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lead", [0, 1, 2, 3, 5, 8, 13])
@pytest.mark.parametrize("pad", [0, 1, 7, 32])
def test_logprobs_alignments(lead, pad, dtype):
    for V in (29, 3001, 17001):
        _check_logprobs(6, V, dtype, stride=V + pad, lead=lead, k=9)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("T", [0.3, 1.0, 3.0])
def test_logprobs_masks(mask, T, dtype):
    for V in (40, 5003, 50257):
        _check_logprobs(4, V, dtype, T=T, mask=mask, k=min(V, 12))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [1, 30, 1111, 20011])
def test_logprobs_rows_that_leave_little(V, dtype):
    """Rows masked throughout, with the lowest value throughout, with one column
    left, constant, and rising or falling by column; fewer columns left than
    alternatives asked for."""
    low = torch.finfo(dtype).min
    z = torch.full((8, V), -math.inf)
    z[1] = low
    z[2, V // 2] = 3.0
    z[3] = 1.5
    z[4] = torch.arange(V) / 64.0
    z[5] = -torch.arange(V) / 64.0
    z[6, :] = -0.0
    z[6, ::2] = 0.0
    z[7] = low
    z[7, V - 1] = 1.0
    targets = torch.tensor([0, V - 1, V // 2, 0, 0, -1, 0, V - 1])
    for k in (1, min(V, 5), min(V, 128)):
        _check_logprobs(8, V, dtype, k=k, z=z, targets=targets)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [33, 5000, 40009])
def test_logprobs_nan_and_infinity(V, dtype):
    z = torch.randn(5, V, generator=torch.Generator().manual_seed(1))
    z[0, V // 3] = math.nan
    z[1, V - 1] = math.inf
    z[2, 0] = -math.inf
    z[3, 5] = math.nan
    z[3, 2] = math.nan
    targets = torch.tensor([1, 1, 1, -1, 4])
    _, view, _, _ = _rows(5, V, V, dtype)
    view.copy_(z.to(dtype))
    lp, ent, lse = _f32(5), _f32(5), _f32(5)
    ids = torch.empty(5, 3, dtype=torch.int32, device=DEV)
    tops = torch.empty(5, 3, dtype=FP32, device=DEV)
    zs.zs_token_logprobs(view, CODE[dtype], 5, V, V, targets.to(DEV), 1.0, lp, ent, lse, 3, ids,
                         tops)
    nan = [torch.isnan(x).tolist() for x in (lp, ent, lse)]
    assert nan[1] == nan[2] == [True, True, False, True, False]
    assert nan[0] == [True, True, False, False, False]   # row 3 has no target
    assert torch.equal(ids.cpu().long(), ref.top(view.cpu().double(), 3))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("k", [1, 2, 31, 64, 127, 128])
def test_top_alternatives(k, dtype):
    """Ties by the thousand (few distinct values), and columns that all fall to
    few threads: the largest values 16, 512, 4096 or 8192 columns apart."""
    g = torch.Generator().manual_seed(k)
    for V in (128, 1500, 30011, 151936):
        z = torch.randint(-4, 5, (4, V), generator=g).float()
        for r, apart in ((1, 16), (2, 512), (3, 4096)):
            z[r] = torch.randn(V, generator=g)
            z[r, ::apart] += 10.0
            z[r, 1::apart] += 10.0
        _check_logprobs(4, V, dtype, k=k, z=z)
    z = torch.zeros(2, 151936)
    for i in range(16):
        z[0, i::8192] = 5.0 + torch.rand(len(range(i, 151936, 8192)), generator=g)
        z[1, i::4096] = 5.0
    _check_logprobs(2, 151936, dtype, k=k, z=z)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_top_alternatives_of_many_rows(dtype):
    """Thousands of rows whose largest values gather in few threads' chunks, so
    that the exact search over the whole table runs in every block."""
    R, V = 2500, 20011
    z = torch.randn(R, V, generator=torch.Generator().manual_seed(2))
    for i in range(16):
        z[:, i::4096] += 8.0
    _check_logprobs(R, V, dtype, k=128, z=z)
    _check_logprobs(R, V, dtype, k=40, z=z)


def test_logprobs_each_output_alone_and_other_streams():
    R, V = 37, 5003
    _, view, z64, g = _rows(R, V, V, BF16)
    targets = _targets(R, V, g).to(DEV)
    full = [_f32(R), _f32(R), _f32(R)]
    zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, targets, 1.0, *full)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(3):
        one = [None, None, None]
        one[i] = _f32(R)
        zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, targets, 1.0, *one, stream=side)
        side.synchronize()
        assert torch.equal(one[i], full[i])
    ids = torch.empty(R, 4, dtype=torch.int32, device=DEV)
    tops = torch.empty(R, 4, dtype=FP32, device=DEV)
    zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, None, 1.0, top_k=4, top_ids=ids,
                         top_logprobs=tops)
    assert torch.equal(ids.cpu().long(), ref.top(z64, 4))


def _upstream(R, g, zero=()):
    x = torch.randn(R, generator=g)
    for r in zero:
        x[r] = 0.0
    return x


def _grad_buffers(R, V, dtype, gstride, glead):
    buf = torch.full((glead + R * gstride + 8,), CANARY, dtype=dtype, device=DEV)
    return buf, torch.as_strided(buf, (R, V), (gstride, 1), glead)


def _assert_untouched(buf, view, R, V, stride, lead):
    keep = torch.ones(buf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(keep, (R, V), (stride, 1), lead).fill_(False)
    assert bool((buf[keep].float() == torch.tensor(CANARY, dtype=buf.dtype).float().item()).all()), \
        "elements outside the gradient were written"


def _check_token_grad(R, V, dtype, T=1.0, stride=None, lead=0, gstride=None, glead=0, mask=None,
                      use=("a", "b"), in_place=False, z=None, targets=None, seed=0):
    stride = stride or V
    gstride = gstride or V
    buf, view, z64, g = _rows(R, V, stride, dtype, lead, seed, mask=mask)
    if z is not None:
        view.copy_(z.to(dtype))
        z64 = view.cpu().double()
    targets = _targets(R, V, g) if targets is None else targets
    o = ref.token_logprobs(z64, targets, T)
    lse, H = o["lse"].float(), o["entropy"].float()
    a = _upstream(R, g, zero=[R - 1]) if "a" in use else None
    b = _upstream(R, g, zero=[R - 1, R // 2]) if "b" in use else None
    if in_place:
        gbuf, gview, gstride, glead = buf, view, stride, lead
    else:
        gbuf, gview = _grad_buffers(R, V, dtype, gstride, glead)
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    zs.zs_token_logprobs_grad(view, CODE[dtype], R, V, stride, targets.to(DEV), T, d(lse), d(H),
                              d(a), d(b), gview, gstride)
    torch.cuda.synchronize()
    want = ref.token_grad(z64, targets, T, lse, H, a, b)
    a64, b64 = ref._weights(a, R).abs(), ref._weights(b, R).abs()
    live = torch.where(torch.isfinite(z64), z64, 0.0).abs().amax(1) / T if mask == "inf" \
        else math.log(V) + 40.0
    coef = (a64 + b64 * (2 * H.double().abs() + 2 * live + 4)) / T
    tol = ref.tol_grad(z64, T, lse, coef, V, dtype == BF16, want, 4 * ref.EPS * a64 / T)
    _assert_within(gview, want, tol, "d_logits")
    _assert_untouched(gbuf, gview, R, V, gstride, glead)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", VOCABS)
def test_token_grad_sizes(V, dtype):
    _check_token_grad(3, V, dtype, T=0.8)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("use", ["a", "b", "ab"])
@pytest.mark.parametrize("R,V", [(1, 50257), (9, 1000), (153, 3001), (2000, 777)])
def test_token_grad_rows(R, V, use, dtype):
    _check_token_grad(R, V, dtype, use=use)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lead,glead", [(0, 0), (1, 1), (3, 0), (0, 5), (7, 2), (8, 16)])
@pytest.mark.parametrize("pad,gpad", [(0, 0), (1, 0), (0, 3), (24, 8)])
def test_token_grad_alignments(lead, glead, pad, gpad, dtype):
    for V in (29, 9001):
        _check_token_grad(5, V, dtype, stride=V + pad, lead=lead, gstride=V + gpad, glead=glead)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("in_place", [False, True])
def test_token_grad_masks_and_in_place(mask, in_place, dtype):
    for V, lead in ((40, 1), (5003, 0), (50257, 3)):
        _check_token_grad(4, V, dtype, T=1.5, mask=mask, in_place=in_place, lead=lead)


def _teacher_record(R, V, K, g, dtype):
    ids = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else
                       torch.randint(0, V, (K,), generator=g) for _ in range(R)]).int()
    t = torch.sort(torch.randn(R, K, generator=g) * 2 + 3, dim=1, descending=True).values.to(dtype)
    if K > 2:
        ids[R // 3, K // 2:] = -1          # a short record
        ids[0, 1] = ids[0, 0]              # a repeated id
        t[R - 1, K - 1] = -math.inf        # an entry without mass
    if R > 3:
        ids[1] = -1                        # no record
    return ids, t


def _check_distill(R, V, K, dtype, T=1.0, tdtype=FP32, own_lse=False, hard=True, stride=None,
                   lead=0, gstride=None, glead=0, mask=None, mode="fused", in_place=False,
                   soft=True, seed=0, z=None):
    """mode: loss (forward alone), grad (from the normalisers) or fused."""
    stride = stride or V
    gstride = gstride or V
    buf, view, z64, g = _rows(R, V, stride, dtype, lead, seed, mask=mask)
    if z is not None:
        view.copy_(z.to(dtype))
        z64 = view.cpu().double()
    ids = t = tl = None
    if K:
        ids, t = _teacher_record(R, V, K, g, tdtype)
        t64 = t.double()
        if own_lse:
            tl = (torch.logsumexp(torch.where(ids >= 0, t64, -50.0) / T, 1) + 0.2).float()
    targets = _targets(R, V, g) if hard else None
    if hard and K:
        targets[0] = int(ids[0, 0])        # the target is among the teacher's ids
    tl64 = None if tl is None else tl.double()
    o = ref.distill(z64, ids, None if t is None else t64, tl64, T, targets)
    w = _upstream(R, g, zero=[R - 1]) if soft and K and mode != "loss" else None
    h = _upstream(R, g, zero=[R - 1]) if hard and mode != "loss" else None
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    head = (view, CODE[dtype], R, V, stride, d(ids), d(t), CODE[tdtype], K, d(tl), T, d(targets))
    loss = _f32(R) if K else None
    lse, logprob, hard_lse = _f32(R), _f32(R) if hard else None, _f32(R)
    if mode != "loss":
        if in_place:
            gbuf, gview, gstride, glead = buf, view, stride, lead
        else:
            gbuf, gview = _grad_buffers(R, V, dtype, gstride, glead)
    in_lse, in_hard = o["lse"].float(), o["hard_lse"].float()
    if mode == "loss":
        zs.zs_distill_loss(*head, loss, lse, logprob, hard_lse)
    elif mode == "grad":
        zs.zs_distill_grad(*head, d(in_lse) if w is not None else None,
                           d(in_hard) if h is not None else None, d(w), d(h), gview, gstride)
    else:
        zs.zs_distill_loss_grad(*head, d(w), d(h), loss, lse, logprob, hard_lse, gview, gstride)
    torch.cuda.synchronize()
    if K:
        q, lnq, at = ref.teacher(ids, t64, tl64, T, V)
    if mode != "grad":
        _assert_within(lse, o["lse"], ref.tol_lse(z64, o["lse"], T), "lse")
        _assert_within(hard_lse, o["hard_lse"], ref.tol_lse(z64, o["hard_lse"], 1.0), "hard_lse")
        if hard:
            _assert_within(logprob, o["logprob"], ref.tol_logprob(z64, o["logprob"], 1.0, V),
                           "logprob")
        if K:
            lnp, _ = ref._masked_log_softmax(z64 / T)
            _assert_within(loss, o["loss"], ref.tol_loss(z64, ids, torch.where(ids >= 0, t64, 0.0),
                                                         tl64, T, lnp.gather(1, at), q, lnq),
                           "loss")
    if mode != "loss":
        exact_lse = mode == "fused"
        want = ref.distill_grad(z64, ids, None if t is None else t64, tl64, T, targets,
                                o["lse"] if exact_lse else in_lse,
                                o["hard_lse"] if exact_lse else in_hard, w, h)
        w64, h64 = ref._weights(w, R).abs(), ref._weights(h, R).abs()
        Q = q.sum(1) if K else torch.zeros(R, dtype=torch.float64)
        tq = ref.tol_q(torch.where(ids >= 0, t64, 0.0), T, tl64) if K else 0.0
        special = w64 / T * (q.amax(1) if K else 0.0) * 2 * tq + 4 * ref.EPS * (h64 + w64 / T * Q)
        tol = ref.tol_grad(z64, T, o["lse"], w64 / T * Q, V, dtype == BF16, want, special)
        tol = tol + ref.tol_grad(z64, 1.0, o["hard_lse"], h64, V, False, torch.zeros_like(want),
                                 torch.zeros(R, dtype=torch.float64))
        tol = tol + (w64 / T * Q * (tq if K else 0.0))[:, None] * \
            torch.nan_to_num((z64 / T - o["lse"][:, None]).exp())
        _assert_within(gview, want, tol, "d_logits")
        _assert_untouched(gbuf, gview, R, V, gstride, glead)


MODES = ["loss", "grad", "fused"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", VOCABS)
def test_distill_sizes(V, dtype, mode):
    _check_distill(4, V, min(V, 16), dtype, T=2.0, mode=mode)
    _check_distill(4, V, min(V, 5), dtype, T=1.0, mode=mode, tdtype=BF16)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("K", [1, 2, 31, 33, 64, 128, 255, 256])
def test_distill_records(K, mode):
    for own_lse in (False, True):
        _check_distill(5, 3001, K, BF16, T=1.5, mode=mode, own_lse=own_lse)
        _check_distill(5, 3001, K, FP32, mode=mode, own_lse=own_lse, tdtype=BF16, hard=False)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("R,V", [(1, 50257), (2, 151936), (9, 1000), (153, 3001), (305, 9000),
                                 (1000, 1000), (1500, 4999)])
def test_distill_rows(R, V, dtype, mode):
    _check_distill(R, V, 8, dtype, mode=mode, T=1.25)


@pytest.mark.parametrize("mode", ["grad", "fused"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lead,glead", [(0, 0), (1, 1), (3, 0), (0, 5), (8, 16)])
@pytest.mark.parametrize("pad,gpad", [(0, 0), (1, 0), (0, 3), (24, 8)])
def test_distill_alignments(lead, glead, pad, gpad, dtype, mode):
    for V in (29, 9001):
        _check_distill(5, V, 6, dtype, mode=mode, stride=V + pad, lead=lead, gstride=V + gpad,
                       glead=glead)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_masks(mask, dtype, mode):
    for V in (40, 5003, 50257):
        _check_distill(4, V, 3, dtype, T=2.0, mask=mask, mode=mode)


@pytest.mark.parametrize("mode", ["grad", "fused"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_in_place_and_parts(dtype, mode):
    for V, lead in ((40, 1), (5003, 0), (50257, 3), (151936, 0)):
        _check_distill(4, V, 12, dtype, T=2.0, mode=mode, in_place=True, lead=lead)
        _check_distill(4, V, 12, dtype, mode=mode, soft=False)
        _check_distill(4, V, 12, dtype, mode=mode, hard=False)
    if mode == "fused":
        _check_distill(4, 5003, 0, dtype, mode=mode)   # cross entropy of the targets alone


@pytest.mark.parametrize("mode", ["grad", "fused"])
@pytest.mark.parametrize("T", [0.05, 20.0])
def test_distill_one_loss_weighted_at_another_temperature(T, mode):
    """Logits of some hundreds, whose exponentials at the other temperature are
    out of range."""
    z = torch.randn(4, 3001, generator=torch.Generator().manual_seed(9)) * 60 + 100
    for dtype in (BF16, FP32):
        _check_distill(4, 3001, 5, dtype, T=T, mode=mode, soft=False, z=z)
        _check_distill(4, 3001, 5, dtype, T=T, mode=mode, hard=False, z=z)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [5, 3000, 20001])
def test_masked_rows_and_unweighted_rows_have_no_gradient(V, dtype):
    """Row 0 is masked throughout; row 1 has weight 0 and NaN logits."""
    R = 3
    _, view, _, g = _rows(R, V, V, dtype)
    view[0] = -math.inf
    view[1] = math.nan
    targets = torch.tensor([1, 2, 3], device=DEV)
    one = torch.tensor([1.0, 0.0, 1.0], device=DEV)
    out = [_f32(R) for _ in range(4)]
    ids = torch.zeros(R, 1, dtype=torch.int32, device=DEV)
    t = torch.zeros(R, 1, device=DEV)
    _, gview = _grad_buffers(R, V, dtype, V, 0)
    zs.zs_distill_loss_grad(view, CODE[dtype], R, V, V, ids, t, zs.ZS_FP32, 1, None, 1.0, targets,
                            one, one, *out, gview, V)
    assert bool((gview[:2] == 0).all()) and bool((gview[2] != 0).any())
    assert out[1][0].item() == -math.inf and out[2][0].item() == -math.inf
    assert out[0][0].item() == math.inf
    gview.fill_(CANARY)
    lse, H = _f32(R), _f32(R)
    zs.zs_token_logprobs(view, CODE[dtype], R, V, V, targets, 1.0, entropy=H, lse=lse)
    assert H[0].item() == 0.0
    zs.zs_token_logprobs_grad(view, CODE[dtype], R, V, V, targets, 1.0, lse, H, one, one, gview, V)
    assert bool((gview[:2] == 0).all()) and bool((gview[2] != 0).any())


def test_ids_out_of_range_are_reported():
    R, V = 4, 5003
    _, view, z64, _ = _rows(R, V, V, BF16)
    targets = torch.tensor([1, V, -1, 1 << 40])
    lp = _f32(R)
    zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, targets.to(DEV), 1.0, lp)
    assert torch.isnan(lp).tolist() == [False, True, False, True]
    with pytest.raises(zs.ZsError) as e:
        zs.zs_check_device_error()
    assert e.value.status == zs.ZS_ERR_RANGE
    zs.zs_check_device_error()                       # cleared
    ids = torch.tensor([[1, V], [2, 3], [1 << 30, 4], [5, -1]], dtype=torch.int32, device=DEV)
    t = torch.zeros(R, 2, device=DEV)
    loss, grad = _f32(R), _grad_buffers(R, V, BF16, V, 0)[1]
    one = torch.ones(R, device=DEV)
    zs.zs_distill_loss_grad(view, zs.ZS_BF16, R, V, V, ids, t, zs.ZS_FP32, 2, None, 1.0, None, one,
                            None, loss, None, None, None, grad, V)
    with pytest.raises(zs.ZsError):
        zs.zs_check_device_error()
    want = ref.distill(z64, ids.cpu(), t.cpu().double(), None, 1.0, None)["loss"]
    _assert_within(loss, want, 1e-4, "loss")


def test_gradients_against_differences():
    """fp32 gradients against central differences of the 64-bit losses."""
    R, V, K, T, h = 3, 19, 4, 1.5, 1e-5
    _, view, z64, g = _rows(R, V, V, FP32)
    targets = torch.tensor([2, 18, -100])
    ids, t = _teacher_record(R, V, K, g, FP32)
    w, a, b = (torch.randn(R, generator=g) for _ in range(3))
    out, gview = [_f32(R) for _ in range(4)], _grad_buffers(R, V, FP32, V, 0)[1]
    zs.zs_distill_loss_grad(view, zs.ZS_FP32, R, V, V, ids.to(DEV), t.to(DEV), zs.ZS_FP32, K, None,
                            T, targets.to(DEV), w.to(DEV), a.to(DEV), *out, gview, V)

    def soft(x):
        o = ref.distill(x, ids, t.double(), None, T, targets)
        return w.double() * o["loss"] + a.double() * o["logprob"]

    def policy(x):
        o = ref.token_logprobs(x, targets, T)
        return a.double() * o["logprob"] + b.double() * o["entropy"]

    def differences(f):
        d = torch.zeros(R, V, dtype=torch.float64)
        for j in range(V):
            up, dn = z64.clone(), z64.clone()
            up[:, j] += h
            dn[:, j] -= h
            d[:, j] = (f(up) - f(dn)) / (2 * h)
        return d

    # fp32 arithmetic on values of order 10: 2^-24 * 10 * the bounds' ~100 roundings
    assert torch.allclose(gview.cpu().double(), differences(soft), rtol=0, atol=1e-4)
    lse, H = _f32(R), _f32(R)
    zs.zs_token_logprobs(view, zs.ZS_FP32, R, V, V, None, T, entropy=H, lse=lse)
    zs.zs_token_logprobs_grad(view, zs.ZS_FP32, R, V, V, targets.to(DEV), T, lse, H, a.to(DEV),
                              b.to(DEV), gview, V)
    assert torch.allclose(gview.cpu().double(), differences(policy), rtol=0, atol=1e-4)


def test_rows_past_32_bit_offsets():
    """Rows 2^31 + 64 elements apart: the third starts past 2^32."""
    R, V, stride = 3, 1003, (1 << 31) + 64
    big = torch.empty(2 * stride + V, dtype=BF16, device=DEV)
    view = torch.as_strided(big, (R, V), (stride, 1))
    z = torch.randn(R, V, generator=torch.Generator().manual_seed(3)).to(BF16)
    view.copy_(z)
    targets = torch.tensor([5, 6, 1002], device=DEV)
    one, out = torch.ones(R, device=DEV), [_f32(R) for _ in range(3)]
    ids = torch.empty(R, 2, dtype=torch.int32, device=DEV)
    tops = torch.empty(R, 2, device=DEV)
    zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, stride, targets, 1.0, *out, 2, ids, tops)
    o = ref.token_logprobs(z.double(), targets.cpu(), 1.0)
    _assert_within(out[0], o["logprob"], ref.tol_logprob(z.double(), o["logprob"], 1.0, V), "lp")
    assert torch.equal(ids.cpu().long(), ref.top(z.double(), 2))
    lse32 = out[2].cpu()
    zs.zs_token_logprobs_grad(view, zs.ZS_BF16, R, V, stride, targets, 1.0, out[2], None, one,
                              None, view, stride)
    want = ref.token_grad(z.double(), targets.cpu(), 1.0, lse32, None, torch.ones(R), None)
    ones = torch.ones(R, dtype=torch.float64)
    _assert_within(view, want, ref.tol_grad(z.double(), 1.0, lse32, ones, V, True, want,
                                            4 * ref.EPS * ones), "d_logits")


@pytest.mark.parametrize("overlap", [0, 1])
def test_same_call_same_bits_and_chained_calls(overlap):
    """Forward, gradient in place and forward again, queued without a wait, three
    times over the same logits: every repetition gives the same bits."""
    R, V, K = 211, 30011, 16
    _, view, z64, g = _rows(R, V, V, BF16)
    keep = view.clone()
    ids, t = _teacher_record(R, V, K, g, FP32)
    ids, t, targets = ids.to(DEV), t.to(DEV), _targets(R, V, g).to(DEV)
    w = torch.randn(R, generator=g).to(DEV)
    old = zs.zs_set_launch_overlap(overlap)
    try:
        runs = []
        for _ in range(3):
            view.copy_(keep)
            o = [_f32(R) for _ in range(8)]
            ti = torch.empty(R, 7, dtype=torch.int32, device=DEV)
            tp = torch.empty(R, 7, device=DEV)
            zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, targets, 1.0, o[0], o[1], o[2], 7, ti,
                                 tp)
            zs.zs_distill_loss_grad(view, zs.ZS_BF16, R, V, V, ids, t, zs.ZS_FP32, K, None, 2.0,
                                    targets, w, w, o[3], o[4], o[5], o[6], view, V)
            zs.zs_token_logprobs(view, zs.ZS_BF16, R, V, V, None, 1.0, lse=o[7])
            runs.append([*o, ti, tp, view.clone()])
        torch.cuda.synchronize()
    finally:
        zs.zs_set_launch_overlap(old)
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
