"""The vocabulary-row losses without a GPU: the 64-bit reference's gradients
against differences of its losses, and what the entry points refuse before
any CUDA call."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import loss_reference as ref

R, V, K = 3, 11, 4


def _data(seed=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(R, V, generator=g, dtype=torch.float64) * 2
    targets = torch.tensor([3, -100, 10])
    ids = torch.tensor([[1, 3, 5, 1], [0, 2, -1, -1], [10, 4, 7, 8]])
    t = torch.randn(R, K, generator=g, dtype=torch.float64)
    return z, targets, ids, t, torch.randn(R, generator=g, dtype=torch.float64)


def _differences(f, z, h=1e-5):
    g = torch.zeros_like(z)
    for r in range(z.shape[0]):
        for j in range(z.shape[1]):
            up, dn = z.clone(), z.clone()
            up[r, j] += h
            dn[r, j] -= h
            g[r, j] = (f(up) - f(dn)) / (2 * h)
    return g


@pytest.mark.parametrize("T", [1.0, 0.7, 2.5])
def test_reference_token_gradient_is_the_difference_quotient(T):
    z, targets, _, _, b = _data()
    a = torch.tensor([0.3, 2.0, -1.1], dtype=torch.float64)

    def total(x):
        o = ref.token_logprobs(x, targets, T)
        return (a * o["logprob"] + b * o["entropy"]).sum()

    o = ref.token_logprobs(z, targets, T)
    g = ref.token_grad(z, targets, T, o["lse"], o["entropy"], a, b)
    # central differences: h^2/6 of the third derivative, and cancellation ~1e-16/h
    assert torch.allclose(g, _differences(total, z), rtol=0, atol=1e-8)


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("own_lse", [False, True])
def test_reference_distill_gradient_is_the_difference_quotient(T, own_lse):
    z, targets, ids, t, w = _data(1)
    h = torch.tensor([0.4, 1.0, -0.2], dtype=torch.float64)
    tl = torch.logsumexp(t / T, 1) + 0.3 if own_lse else None

    def total(x):
        o = ref.distill(x, ids, t, tl, T, targets)
        return (w * o["loss"] + h * o["logprob"]).sum()

    o = ref.distill(z, ids, t, tl, T, targets)
    g = ref.distill_grad(z, ids, t, tl, T, targets, o["lse"], o["hard_lse"], w, h)
    assert torch.allclose(g, _differences(total, z), rtol=0, atol=1e-8)


def test_reference_top_breaks_ties_by_id():
    z = torch.tensor([[1.0, 3.0, 3.0, -math.inf, math.nan, 0.0, -0.0]], dtype=torch.float64)
    assert ref.top(z, 7).tolist() == [[4, 1, 2, 0, 5, 6, 3]]


# ---------------------------------------------------------------- refusals ----
BUF = np.zeros(1 << 12, np.uint8)
P = BUF.ctypes.data + (-BUF.ctypes.data) % 16   # an aligned host address


def _status(call):
    with pytest.raises(zs.ZsError) as e:
        call()
    return e.value.status


def _logprobs(logits=P, dtype=zs.ZS_FP32, rows=1, vocab=8, stride=8, targets=P + 64, T=1.0,
              logprob=P + 128, entropy=None, lse=None, top_k=0, ids=None, top=None):
    zs.zs_token_logprobs(logits, dtype, rows, vocab, stride, targets, T, logprob, entropy, lse,
                         top_k, ids, top, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=zs.ZS_FP24), zs.ZS_ERR_INVAL), (dict(dtype=9), zs.ZS_ERR_INVAL),
    (dict(logits=None), zs.ZS_ERR_INVAL), (dict(targets=None), zs.ZS_ERR_INVAL),
    (dict(logprob=None), zs.ZS_ERR_INVAL), (dict(rows=-1), zs.ZS_ERR_RANGE),
    (dict(rows=1 << 31), zs.ZS_ERR_RANGE), (dict(vocab=0, stride=0), zs.ZS_ERR_RANGE),
    (dict(vocab=zs.ZS_MAX_VOCAB + 1, stride=1 << 21), zs.ZS_ERR_RANGE),
    (dict(stride=7), zs.ZS_ERR_RANGE), (dict(stride=1 << 41), zs.ZS_ERR_RANGE),
    (dict(T=0.0), zs.ZS_ERR_INVAL), (dict(T=-1.0), zs.ZS_ERR_INVAL),
    (dict(T=math.inf), zs.ZS_ERR_INVAL), (dict(T=math.nan), zs.ZS_ERR_INVAL),
    (dict(T=1e-60), zs.ZS_ERR_INVAL), (dict(T=1e60), zs.ZS_ERR_INVAL),
    (dict(top_k=-1), zs.ZS_ERR_RANGE), (dict(top_k=9), zs.ZS_ERR_RANGE),
    (dict(top_k=zs.ZS_MAX_TOP + 1, vocab=1000, stride=1000), zs.ZS_ERR_RANGE),
    (dict(top_k=2, ids=P + 256), zs.ZS_ERR_INVAL), (dict(top_k=2, top=P + 256), zs.ZS_ERR_INVAL),
    (dict(logits=P + 2), zs.ZS_ERR_ALIGN), (dict(targets=P + 68), zs.ZS_ERR_ALIGN),
    (dict(logprob=P + 129), zs.ZS_ERR_ALIGN), (dict(lse=P + 130), zs.ZS_ERR_ALIGN),
    (dict(logprob=P + 28), zs.ZS_ERR_INVAL),          # an output inside the logits
    (dict(entropy=P + 128), zs.ZS_ERR_INVAL),         # two outputs in one place
    (dict(), zs.ZS_ERR_INVAL),                        # host memory
])
def test_token_logprobs_refuses(change, status):
    assert _status(lambda: _logprobs(**change)) == status


def _logprobs_grad(logits=P, dtype=zs.ZS_FP32, rows=2, vocab=8, stride=8, targets=P + 64, T=1.0,
                   lse=P + 128, entropy=P + 144, a=P + 160, b=P + 176, out=P + 256, ostride=8):
    zs.zs_token_logprobs_grad(logits, dtype, rows, vocab, stride, targets, T, lse, entropy, a, b,
                              out, ostride, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(out=None), zs.ZS_ERR_INVAL), (dict(lse=None), zs.ZS_ERR_INVAL),
    (dict(a=None, b=None), zs.ZS_ERR_INVAL), (dict(targets=None), zs.ZS_ERR_INVAL),
    (dict(entropy=None), zs.ZS_ERR_INVAL), (dict(ostride=7), zs.ZS_ERR_RANGE),
    (dict(out=P + 258), zs.ZS_ERR_ALIGN), (dict(out=P + 32), zs.ZS_ERR_INVAL),
    (dict(out=P, ostride=9), zs.ZS_ERR_INVAL),        # in place needs the same stride
    (dict(out=P), zs.ZS_ERR_INVAL),                   # in place, but host memory
    (dict(dtype=zs.ZS_FP24), zs.ZS_ERR_INVAL), (dict(T=0.0), zs.ZS_ERR_INVAL),
])
def test_token_logprobs_grad_refuses(change, status):
    assert _status(lambda: _logprobs_grad(**change)) == status


ROWS = dict(logits=P, dtype=zs.ZS_FP32, rows=2, vocab=8, stride=8, ids=P + 64, t=P + 96,
            tdtype=zs.ZS_FP32, k=2, tlse=P + 112, T=1.0, targets=P + 128, w=P + 144, h=P + 152,
            loss=P + 160, lse=P + 168, logprob=P + 176, hard_lse=P + 184, out=P + 256, ostride=8)


def _distill(kind, **change):
    a = dict(ROWS, **change)
    head = [a[x] for x in ("logits", "dtype", "rows", "vocab", "stride", "ids", "t", "tdtype",
                           "k", "tlse", "T", "targets")]
    if kind == "loss":
        zs.zs_distill_loss(*head, a["loss"], a["lse"], a["logprob"], a["hard_lse"], stream=0)
    elif kind == "grad":
        zs.zs_distill_grad(*head, a["lse"], a["hard_lse"], a["w"], a["h"], a["out"], a["ostride"],
                           stream=0)
    else:
        zs.zs_distill_loss_grad(*head, a["w"], a["h"], a["loss"], a["lse"], a["logprob"],
                                a["hard_lse"], a["out"], a["ostride"], stream=0)


@pytest.mark.parametrize("kind", ["loss", "grad", "loss_grad"])
@pytest.mark.parametrize("change,status", [
    (dict(k=-1), zs.ZS_ERR_RANGE), (dict(k=zs.ZS_MAX_TEACHER + 1), zs.ZS_ERR_RANGE),
    (dict(k=0), zs.ZS_ERR_INVAL), (dict(ids=None), zs.ZS_ERR_INVAL),
    (dict(t=None), zs.ZS_ERR_INVAL), (dict(tdtype=zs.ZS_FP24), zs.ZS_ERR_INVAL),
    (dict(ids=P + 66), zs.ZS_ERR_ALIGN), (dict(tlse=P + 114), zs.ZS_ERR_ALIGN),
    (dict(targets=None), zs.ZS_ERR_INVAL), (dict(T=math.nan), zs.ZS_ERR_INVAL),
    (dict(stride=5), zs.ZS_ERR_RANGE), (dict(logits=None), zs.ZS_ERR_INVAL),
    (dict(), zs.ZS_ERR_INVAL),                        # host memory
])
def test_distill_refuses(kind, change, status):
    assert _status(lambda: _distill(kind, **change)) == status


@pytest.mark.parametrize("kind,change,status", [
    ("loss", dict(loss=None, lse=None, logprob=None, hard_lse=None), zs.ZS_ERR_INVAL),
    ("loss", dict(loss=P + 100), zs.ZS_ERR_INVAL),    # an output inside the teacher's logits
    ("grad", dict(lse=None), zs.ZS_ERR_INVAL), ("grad", dict(hard_lse=None), zs.ZS_ERR_INVAL),
    ("grad", dict(w=None, h=None), zs.ZS_ERR_INVAL), ("grad", dict(out=None), zs.ZS_ERR_INVAL),
    ("loss_grad", dict(out=None), zs.ZS_ERR_INVAL),
    ("loss_grad", dict(w=None, h=None), zs.ZS_ERR_INVAL),
    ("loss_grad", dict(out=P + 4), zs.ZS_ERR_INVAL),
    ("loss_grad", dict(ostride=3), zs.ZS_ERR_RANGE),
])
def test_distill_refuses_more(kind, change, status):
    assert _status(lambda: _distill(kind, **change)) == status


def test_no_rows_is_no_work():
    _logprobs(rows=0, logits=None)
    _logprobs_grad(rows=0, logits=None)
    for kind in ("loss", "grad", "loss_grad"):
        _distill(kind, rows=0, logits=None)


def test_binding_refuses_short_and_strided_buffers():
    z = torch.zeros(4, 10)
    out = torch.zeros(4)
    tgt = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="logits holds"):
        zs.zs_token_logprobs(z, zs.ZS_FP32, 5, 10, 10, None, lse=torch.zeros(5), stream=0)
    with pytest.raises(ValueError, match="dense rows"):
        zs.zs_token_logprobs(z.t(), zs.ZS_FP32, 4, 4, 10, None, lse=out, stream=0)
    with pytest.raises(ValueError, match="dense rows"):
        zs.zs_token_logprobs(z[:, :8], zs.ZS_FP32, 4, 8, 8, None, lse=out, stream=0)
    with pytest.raises(ValueError, match="the call needs"):
        zs.zs_token_logprobs(z[:, :8], zs.ZS_FP32, 4, 9, 10, None, lse=out, stream=0)
    with pytest.raises(ValueError, match="lse holds"):
        zs.zs_token_logprobs(z, zs.ZS_FP32, 4, 10, 10, None, lse=out[:3], stream=0)
    with pytest.raises(ValueError, match="targets holds"):
        zs.zs_token_logprobs(z, zs.ZS_FP32, 4, 10, 10, tgt.int(), logprob=out, stream=0)
    with pytest.raises(ValueError, match="top_ids holds"):
        zs.zs_token_logprobs(z, zs.ZS_FP32, 4, 10, 10, None, top_k=3, top_ids=tgt.int(),
                             top_logprobs=torch.zeros(12), stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        zs.zs_token_logprobs(z, zs.ZS_FP32, 2, 10, 10, None, lse=out[::2], stream=0)
    with pytest.raises(ValueError, match="teacher_logits holds"):
        zs.zs_distill_loss(z, zs.ZS_FP32, 4, 10, 10, torch.zeros(4, 2, dtype=torch.int32),
                           torch.zeros(4, 1), zs.ZS_FP32, 2, None, 1.0, loss=out, stream=0)
