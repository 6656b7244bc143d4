"""The losses over vocabulary rows where a value leaves the usual range: scaled
logits past fp32's, teachers without mass, ids out of range beside the checks of
the bounds-checked build, tokens the model is all but sure of, and losses without
a teacher."""
import math

import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import loss_reference as ref
from gpu_util import DEV
from test_gpu_losses import _check_distill

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: zs.ZS_BF16, torch.float32: zs.ZS_FP32}
BF16, FP32 = torch.bfloat16, torch.float32


def _f32(R):
    return torch.full((R,), 777.0, dtype=FP32, device=DEV)


# ---- scaled logits past fp32's range ---------------------------------------------
def _lowest_rows(V, dtype):
    """Rows whose largest logit is the type's lowest value: everywhere, in half of
    the columns (the others masked), and in one; the ids of a teacher's record and
    the target of each, among the columns that are left."""
    z = torch.full((3, V), torch.finfo(dtype).min, dtype=dtype)
    z[1, V // 2:] = -math.inf
    z[2, 1:] = -math.inf
    ids = torch.tensor([[V - 1, 0, 2], [1, V // 2 - 1, -1], [0, -1, -1]], dtype=torch.int32)
    return z, ids, torch.tensor([2, 1, 0])


def _lowest_gradients(z, ids, t, targets, w, h, T):
    """(of the soft loss, of the hard labels): p is uniform over what is left."""
    p = (~torch.isneginf(z)).double()
    p = p / p.sum(1, keepdim=True)
    q = torch.softmax(torch.where(ids >= 0, t.double() / T, -math.inf), 1)
    soft = (w.double() / T)[:, None] * p
    soft.scatter_add_(1, ids.clamp(min=0).long(), -(w.double() / T)[:, None] * q)
    hard = -h.double()[:, None] * p
    hard.scatter_add_(1, targets[:, None], h.double()[:, None])
    return soft, hard


def _within(got, want, rel, scale, bf16):
    """rel of what the terms add up from, and a bf16 result's own rounding."""
    tol = rel * scale + (want.abs() * ref.BF16_ROUNDING if bf16 else 0.0)
    got = got.detach().cpu().double()
    assert bool(((got - want).abs() <= tol).all()), (got - want).abs().max()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [5, 1000, 50257])
@pytest.mark.parametrize("T", [0.3, 0.7])
def test_rows_of_the_lowest_value_sharpened(T, V, dtype):
    """The lowest value over T < 1 is past fp32's range, so is the row's lse; its
    probabilities, losses and gradients are not."""
    z, ids, targets = _lowest_rows(V, dtype)
    t = torch.tensor([[1.0, 0.5, -1.0], [2.0, 0.0, 9.0], [0.0, 9.0, 9.0]])
    w, h = torch.tensor([0.5, 2.0, 1.0]), torch.tensor([-0.25, 1.0, -3.0])
    R, out = 3, [_f32(3) for _ in range(4)]
    grad = torch.empty(R, V, dtype=dtype, device=DEV)
    head = (z.to(DEV), CODE[dtype], R, V, V, ids.to(DEV), t.to(DEV), zs.ZS_FP32, 3, None, T,
            targets.to(DEV))
    zs.zs_distill_loss_grad(*head, w.to(DEV), h.to(DEV), *out, grad, V)
    soft, hard = _lowest_gradients(z, ids, t, targets, w, h, T)
    # sums and quotients of equal terms: tol_sum's roundings and some 16 more
    rel = ref.tol_sum(V) + 32 * ref.EPS
    scale = (w / T + h.abs()).double()[:, None] * 2
    _within(grad, soft + hard, rel, scale, dtype == BF16)
    loss, lse, logprob, hard_lse = out
    assert bool(torch.isneginf(lse).all()) and bool(torch.isfinite(hard_lse).all())
    live = (~torch.isneginf(z)).sum(1).double()
    _within(logprob, -live.log(), rel, 2 * live.log()[:, None].amax() + 1, False)
    q = torch.softmax(torch.where(ids >= 0, t.double() / T, -math.inf), 1)
    want = torch.where(q > 0, q * (torch.where(q > 0, q, 1.0).log() + live.log()[:, None]), 0.0)
    _within(loss, want.sum(1), rel, 2 * live.log().amax() + 8, False)


# ---- teachers without mass -------------------------------------------------------
@pytest.mark.parametrize("K", [1, 5, 200])
def test_teacher_rows_masked_throughout_have_no_loss(K):
    """A teacher's row masked throughout has lse = -infinity: its record, unused
    entries or entries of -infinity, adds nothing to the loss or the gradient."""
    R, V = 4, 3001
    g = torch.Generator().manual_seed(K)
    z = torch.randn(R, V, generator=g)
    ids = torch.randint(0, V, (R, K), generator=g, dtype=torch.int32)
    t = torch.randn(R, K, generator=g)
    ids[0] = -1
    t[1] = -math.inf
    ids[2] = -1
    lse = torch.tensor([-math.inf, -math.inf, math.nan, 9.0])   # (row 2: of a row not recorded)
    targets = torch.randint(0, V, (R,), generator=g)
    one = torch.ones(R, device=DEV)
    d = lambda x: x.to(DEV)  # noqa: E731
    head = (d(z), zs.ZS_FP32, R, V, V, d(ids), d(t), zs.ZS_FP32, K, d(lse), 1.0, d(targets))
    own, grad = _f32(R), torch.empty(R, V, device=DEV)
    loss, lse_s, hard_lse = _f32(R), _f32(R), _f32(R)
    zs.zs_distill_loss(*head, own, lse_s, None, hard_lse)
    zs.zs_distill_loss_grad(*head, one, one, loss, None, None, None, grad, V)
    alone = torch.empty_like(grad)
    zs.zs_distill_grad(*head, lse_s, hard_lse, one, one, alone, V)
    assert loss[:3].tolist() == own[:3].tolist() == [0.0, 0.0, 0.0]
    assert bool(torch.isfinite(loss[3])) and torch.equal(loss, own)
    p = torch.softmax(z.double(), 1)
    want = -p
    want.scatter_add_(1, targets[:, None], torch.ones(R, 1, dtype=torch.float64))
    rel = ref.tol_sum(V) + 64 * ref.EPS    # of p <= 1, and of the normalisers' size (about 8)
    for got in (grad, alone):
        _within(got[:3], want[:3], rel, 1.0, False)


# ---- ids out of range --------------------------------------------------------------
def test_ids_out_of_range_are_told_from_failed_bounds_checks():
    R, V = 2, 100
    z = torch.zeros(R, V, device=DEV)
    zs.zs_check_device_error()
    zs.zs_token_logprobs(z, zs.ZS_FP32, R, V, V, torch.tensor([1, V], device=DEV), 1.0, _f32(R))
    with pytest.raises(zs.ZsError, match="token id") as e:
        zs.zs_check_device_error()
    assert e.value.status == zs.ZS_ERR_RANGE
    assert "bounds check" not in str(e.value)
    ids = torch.tensor([[0, 1], [2, V]], dtype=torch.int32, device=DEV)
    zs.zs_distill_loss(z, zs.ZS_FP32, R, V, V, ids, torch.zeros(R, 2, device=DEV), zs.ZS_FP32, 2,
                       None, 1.0, None, _f32(R))
    with pytest.raises(zs.ZsError, match="token id") as e:
        zs.zs_check_device_error()
    assert "bounds check" not in str(e.value)
    zs.zs_check_device_error()   # read and cleared


# ---- tokens the model is all but sure of -------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("R", [3, 200])
def test_likely_tokens_keep_their_small_values(R, T, dtype):
    """Two logits left of a row, the likely one behind the other in the same
    thread's share (every block size divides 256 chunks) and 4.5 to 5.5 T above.

    Bounds: with the sums relative to the maximum, S = 1 + x, x = e^-d: one rounding
    of S (EPS), x itself to (3 d / ln 2 + 4) EPS, ln S to EPS of its size; U = -x d /
    ln 2 has x's error and two roundings, the entropy one more of its own size."""
    V, chunk = 32000, 32 // torch.finfo(dtype).bits * 8
    low, high = 16 * chunk, (16 + 256) * chunk
    z = torch.full((R, V), -math.inf)
    z[:, low] = torch.arange(R) / R
    z[:, high] = z[:, low] + T * (4.5 + torch.rand(R, generator=torch.Generator().manual_seed(4)))
    z = z.to(dtype)
    logprob, H, lse = _f32(R), _f32(R), _f32(R)
    top = torch.empty(R, 2, device=DEV)
    ids = torch.empty(R, 2, dtype=torch.int32, device=DEV)
    target = torch.full((R,), high, dtype=torch.int64, device=DEV)
    zs.zs_token_logprobs(z.to(DEV), CODE[dtype], R, V, V, target, T, logprob, H, lse, 2, ids, top)
    d = ((z[:, high].double() - z[:, low].double()) / T)
    x = torch.exp(-d)
    ln_s = torch.log1p(x)
    each = (3 * d / math.log(2) + 4) * ref.EPS
    tol = ref.EPS * (1 + 2 * ln_s) + x * each
    assert bool(((logprob.cpu().double() + ln_s).abs() <= tol).all())
    assert bool(((top[:, 0].cpu().double() + ln_s).abs() <= tol).all())
    want = ln_s + x * d / (1 + x)
    tol = tol + x * d * (each + 4 * ref.EPS) + ref.EPS * want
    assert bool(((H.cpu().double() - want).abs() <= tol).all())


# ---- no teacher --------------------------------------------------------------------
@pytest.mark.parametrize("mode", ["loss", "grad", "fused"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("R,V", [(1, 1), (5, 33), (700, 1000), (153, 4099), (3, 50257),
                                 (2, 151936), (200, 90001)])
def test_cross_entropy_without_a_teacher(R, V, dtype, mode):
    _check_distill(R, V, 0, dtype, mode=mode)
    _check_distill(R, V, 0, dtype, T=1.5, mode=mode, in_place=mode != "loss", mask="lowest")
