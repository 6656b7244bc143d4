"""The operators around the layers without a GPU: their 64-bit reference against
differences, and every refusal of the entry points before any CUDA call."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import layers_reference as ref


def _differences(f, x, h=1e-6):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        at = x.reshape(-1)[i].item()
        x.reshape(-1)[i] = at + h
        up = f(x).item()
        x.reshape(-1)[i] = at - h
        g.reshape(-1)[i] = (up - f(x).item()) / (2 * h)
        x.reshape(-1)[i] = at
    return g


def test_reference_layer_norm_gradient_is_the_slope():
    g = torch.Generator().manual_seed(0)
    x, dy, past = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(7, generator=g, dtype=torch.float64) for _ in range(2))

    def total(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-3)["y"] * dy).sum() + (x * past).sum()

    st = ref.layer_norm(x, w, b, 1e-3)
    got = ref.layer_norm_grad(dy, x, w, st["mean"], st["rstd"], past)
    for name, at in (("d_x", x), ("d_weight", w), ("d_bias", b)):
        f = {"d_x": lambda v: total(v, w, b), "d_weight": lambda v: total(x, v, b),
             "d_bias": lambda v: total(x, w, v)}[name]
        assert torch.allclose(got[name], _differences(f, at), rtol=0, atol=1e-7), name


def test_reference_embedding_gradient_is_the_slope():
    g = torch.Generator().manual_seed(1)
    table = torch.randn(5, 3, generator=g, dtype=torch.float64)
    d = torch.randn(6, 3, generator=g, dtype=torch.float64)
    tokens = torch.tensor([4, 0, -1, 4, 4, 1])
    got, _ = ref.embedding_grad(d, tokens, 5, 1.7, None)
    slope = _differences(lambda t: (ref.embedding(t, tokens, 1.7) * d).sum(), table)
    assert torch.allclose(got, slope, rtol=0, atol=1e-7)


# ---------------------------------------------------------------- refusals ----
BUF = np.zeros(1 << 16, np.uint8)
P = BUF.ctypes.data + (-BUF.ctypes.data) % 16   # an aligned host address
F, B = zs.ZS_FP32, zs.ZS_BF16
INVAL, RANGE, ALIGN = zs.ZS_ERR_INVAL, zs.ZS_ERR_RANGE, zs.ZS_ERR_ALIGN


def _status(call):
    with pytest.raises(zs.ZsError) as e:
        call()
    return e.value.status


# (a table of 4 x 8 at 0, tokens of 2 at 512, two rows at 1024, scratch at 4096)
def _embedding(table=P, td=F, vocab=4, dim=8, ts=8, tokens=P + 512, rows=2, scale=1.0,
               out=P + 1024, od=F, os=8):
    zs.zs_embedding(table, td, vocab, dim, ts, tokens, rows, scale, out, od, os, stream=0)


SIZES = [
    (dict(td=zs.ZS_FP24), INVAL), (dict(td=7), INVAL), (dict(rows=-1), RANGE),
    (dict(rows=1 << 31), RANGE), (dict(vocab=0), RANGE), (dict(vocab=zs.ZS_MAX_VOCAB + 1), RANGE),
    (dict(dim=0), RANGE), (dict(dim=zs.ZS_MAX_DIM + 1, ts=1 << 17, os=1 << 17), RANGE),
    (dict(ts=7), RANGE), (dict(os=7), RANGE), (dict(ts=(1 << 40) + 1), RANGE),
    (dict(os=(1 << 40) + 1), RANGE), (dict(rows=(1 << 31) - 1, os=1 << 20), RANGE),
    (dict(vocab=1 << 20, ts=1 << 30), RANGE),
    (dict(scale=math.inf), INVAL), (dict(scale=math.nan), INVAL), (dict(scale=1e39), INVAL),
    (dict(tokens=None), INVAL), (dict(tokens=P + 516), ALIGN), (dict(), INVAL),
]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(od=9), INVAL), (dict(table=None), INVAL), (dict(out=None), INVAL),
    (dict(table=P + 2), ALIGN), (dict(out=P + 1026), ALIGN), (dict(out=P + 124), INVAL),
    (dict(out=P + 512 - 64 + 4), INVAL),
])
def test_embedding_refuses(change, status):
    assert _status(lambda: _embedding(**change)) == status


def _embedding_grad(d_out=P + 1024, od=F, rows=2, dim=8, os=8, tokens=P + 512, vocab=4, scale=1.0,
                    add=P + 2048, ws=P + 4096, ws_bytes=None, d_table=P, td=F, ts=8):
    need = zs.zs_embedding_grad_workspace_bytes(rows, dim) if ws_bytes is None else ws_bytes
    zs._check(zs.lib().zs_embedding_grad(d_out, od, rows, dim, os, tokens, vocab, scale, add, ws,
                                         need, d_table, td, ts, None))


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(od=9), INVAL), (dict(d_out=None), INVAL), (dict(d_table=None), INVAL),
    (dict(ws=None), INVAL), (dict(ws=P + 4100), ALIGN), (dict(ws_bytes=64), RANGE),
    (dict(add=P + 4), INVAL), (dict(add=P + 2050), ALIGN), (dict(d_table=P + 1020), INVAL),
    (dict(d_table=P + 4096), INVAL), (dict(add=P), INVAL),   # in place, but host memory
    (dict(rows=0, d_table=None), INVAL),
])
def test_embedding_grad_refuses(change, status):
    assert _status(lambda: _embedding_grad(**change)) == status


def _layer_norm(x=P, dt=F, rows=2, dim=8, rs=8, residual=P + 256, weight=P + 512, bias=P + 576,
                wd=F, eps=1e-5, total=P + 1024, y=P + 1280, os=8, mean=P + 2048, rstd=P + 2056):
    zs.zs_layer_norm(x, dt, rows, dim, rs, residual, weight, bias, wd, eps, total, y, os, mean,
                     rstd, stream=0)


ROWS = [
    (dict(dt=zs.ZS_FP24), INVAL), (dict(wd=zs.ZS_FP24), INVAL), (dict(rows=-1), RANGE),
    (dict(rows=1 << 31), RANGE), (dict(dim=0), RANGE),
    (dict(dim=zs.ZS_MAX_DIM + 1, rs=1 << 17, os=1 << 17), RANGE), (dict(rs=7), RANGE),
    (dict(os=7), RANGE), (dict(rows=(1 << 31) - 1, rs=1 << 20, os=8), RANGE),
    (dict(x=None), INVAL), (dict(x=P + 2), ALIGN), (dict(weight=P + 514), ALIGN),
    (dict(mean=P + 2050), ALIGN), (dict(rstd=P + 2049), ALIGN), (dict(), INVAL),
]


@pytest.mark.parametrize("change,status", ROWS + [
    (dict(eps=0.0), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=math.nan), INVAL),
    (dict(eps=math.inf), INVAL), (dict(eps=1e-40), INVAL),
    (dict(residual=None), INVAL),                    # sum_out without a residual
    (dict(y=None), INVAL), (dict(bias=P + 577), ALIGN), (dict(y=P + 1282), ALIGN),
    (dict(y=P + 1028), INVAL),                       # y over sum_out
    (dict(y=P + 4), INVAL),                          # y inside x
    (dict(y=P, os=9), INVAL),                        # in place needs one stride
    (dict(y=P), INVAL), (dict(total=P + 256), INVAL),   # in place, but host memory
    (dict(total=P + 256, y=P + 256), INVAL),         # two outputs in one place
    (dict(mean=P + 1024), INVAL), (dict(mean=P + 2056), INVAL), (dict(y=P + 512), INVAL),
])
def test_layer_norm_refuses(change, status):
    assert _status(lambda: _layer_norm(**change)) == status


def _layer_norm_grad(dy=P + 256, x=P, dt=F, rows=2, dim=8, os=8, rs=8, weight=P + 512, wd=F,
                     mean=P + 2048, rstd=P + 2056, past=P + 768, ws=P + 4096, ws_bytes=1 << 14,
                     dx=P + 1024, dw=P + 2560, db=P + 2624, gd=F):
    zs._check(zs.lib().zs_layer_norm_grad(dy, x, dt, rows, dim, os, rs, weight, wd, mean, rstd,
                                          past, ws, ws_bytes, dx, dw, db, gd, None))


@pytest.mark.parametrize("change,status", ROWS + [
    (dict(gd=zs.ZS_FP24), INVAL), (dict(dy=None), INVAL), (dict(mean=None), INVAL),
    (dict(rstd=None), INVAL), (dict(dx=None), INVAL), (dict(ws=None), INVAL),
    (dict(ws=P + 4104), ALIGN), (dict(ws_bytes=8), RANGE), (dict(dw=P + 2562), ALIGN),
    (dict(dx=P), INVAL),                             # d_x in place of x
    (dict(dx=P + 260), INVAL), (dict(dx=P + 256), INVAL),   # in place, but host memory
    (dict(dw=P + 2624), INVAL), (dict(dw=P + 4096), INVAL), (dict(dx=P + 768 - 4), INVAL),
    (dict(rows=0, dw=P + 2562), ALIGN),
])
def test_layer_norm_grad_refuses(change, status):
    assert _status(lambda: _layer_norm_grad(**change)) == status


def _array(kind, values):
    import ctypes
    return (kind * max(len(values), 1))(*values)


def _list(kind="clip", p=(P, P + 256), n=(8, 8), count=None, dt=F, out=(P + 512, P + 768), od=F,
          ws=P + 4096, ws_bytes=None, max_norm=1.0, norm=P + 3328, coef=P + 3336, bad=P + 3344,
          sq=P + 3352):
    import ctypes
    L = zs.lib()
    p = None if p is None else _array(ctypes.c_void_p, p)
    out = None if out is None else _array(ctypes.c_void_p, out)
    lengths = None if n is None else _array(ctypes.c_int64, n)
    count = len(n) if count is None else count
    need = L.zs_grad_norm_workspace_bytes() if ws_bytes is None else ws_bytes
    if kind == "clip":
        st = L.zs_tensors_clip(p, lengths, count, dt, max_norm, out, od, ws, need, norm, coef, bad,
                               None)
    elif kind == "sqnorm":
        st = L.zs_tensors_sqnorm(p, lengths, count, dt, ws, need, sq, None)
    else:
        st = L.zs_tensors_scale(p, lengths, count, dt, coef, bad, out, od, None)
    zs._check(st)


@pytest.mark.parametrize("kind", ["clip", "sqnorm", "scale"])
@pytest.mark.parametrize("change,status", [
    (dict(dt=zs.ZS_FP24), INVAL), (dict(count=-1), RANGE),
    (dict(count=zs.ZS_MAX_TENSORS + 1), RANGE), (dict(n=(8, -1)), RANGE),
    (dict(n=(8, (1 << 44) + 1)), RANGE), (dict(n=(1 << 43, (1 << 43) + 1)), RANGE),
    (dict(n=None, count=2), INVAL), (dict(p=None), INVAL), (dict(p=(P, None)), INVAL),
    (dict(p=(P, P + 258)), ALIGN), (dict(), INVAL),
])
def test_lists_refuse(kind, change, status):
    assert _status(lambda: _list(kind, **change)) == status


@pytest.mark.parametrize("kind", ["clip", "scale"])
@pytest.mark.parametrize("change,status", [
    (dict(od=zs.ZS_FP24), INVAL), (dict(out=None), INVAL), (dict(out=(P + 512, None)), INVAL),
    (dict(out=(P + 512, P + 770)), ALIGN), (dict(coef=None), INVAL),
    (dict(out=(P + 512, P + 516)), INVAL),            # two outputs
    (dict(out=(P + 768, P + 764)), INVAL),            # the same, not in order
    (dict(out=(P + 4, P + 768)), INVAL),              # inside its own input
    (dict(out=(P + 256, P + 512)), INVAL),            # another's input
    (dict(out=(P, P + 256), od=B), INVAL),            # in place needs one dtype
    (dict(out=(P, P + 256)), INVAL),                  # in place, but host memory
    (dict(out=(P + 512, P + 3328)), INVAL),           # the coefficient
])
def test_lists_refuse_outs(kind, change, status):
    assert _status(lambda: _list(kind, **change)) == status


@pytest.mark.parametrize("kind,change,status", [
    ("clip", dict(max_norm=0.0), INVAL), ("clip", dict(max_norm=math.inf), INVAL),
    ("clip", dict(max_norm=math.nan), INVAL), ("clip", dict(norm=None), INVAL),
    ("clip", dict(bad=None), INVAL), ("clip", dict(ws=None), INVAL),
    ("clip", dict(ws=P + 4100), ALIGN), ("clip", dict(ws_bytes=16), RANGE),
    ("clip", dict(norm=P + 3336), INVAL), ("clip", dict(norm=P + 3330), ALIGN),
    ("clip", dict(norm=P + 4), INVAL), ("clip", dict(ws=P), INVAL),
    ("sqnorm", dict(sq=None), INVAL), ("sqnorm", dict(sq=P + 3348), ALIGN),
    ("sqnorm", dict(sq=P + 8), INVAL), ("sqnorm", dict(ws_bytes=0), RANGE),
    ("scale", dict(coef=P + 3337), ALIGN), ("scale", dict(bad=P + 3337), ALIGN),
])
def test_lists_refuse_more(kind, change, status):
    assert _status(lambda: _list(kind, **change)) == status


def test_no_rows_is_no_work():
    _embedding(rows=0, tokens=None, out=None, table=None)
    _layer_norm(rows=0, x=None)
    _layer_norm_grad(rows=0, x=None, dw=None, db=None)
    _list("scale", p=(), n=(), out=())
    _list("scale", p=(None,), n=(0,), out=(None,))


def test_workspace_sizes():
    assert zs.zs_embedding_grad_workspace_bytes(-1, 8) == -1
    assert zs.zs_embedding_grad_workspace_bytes(1, zs.ZS_MAX_DIM + 1) == -1
    assert zs.zs_layer_norm_grad_workspace_bytes(1 << 31, 8) == -1
    assert zs.zs_layer_norm_grad_workspace_bytes(1, 0) == -1
    assert zs.zs_layer_norm_grad_workspace_bytes(1, 8) > 0
    # grows with the tokens, and stays within int64 at the largest sizes
    sizes = [zs.zs_embedding_grad_workspace_bytes(r, zs.ZS_MAX_DIM)
             for r in (1, 1000, 1 << 20, (1 << 31) - 1)]
    assert 0 < sizes[0] < sizes[1] < sizes[2] < sizes[3]


def test_binding_refuses_short_and_strided_buffers():
    t, tok, out = torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="table holds"):
        zs.zs_embedding(t, F, 5, 8, 8, tok, 2, 1.0, out, F, 8, stream=0)
    with pytest.raises(ValueError, match="tokens holds"):
        zs.zs_embedding(t, F, 4, 8, 8, tok.int(), 2, 1.0, out, F, 8, stream=0)
    with pytest.raises(ValueError, match="out holds"):
        zs.zs_embedding(t, F, 4, 8, 8, tok, 2, 1.0, out[:1], F, 8, stream=0)
    with pytest.raises(ValueError, match="dense rows"):
        zs.zs_embedding(t.t(), F, 8, 4, 8, tok, 2, 1.0, out, F, 8, stream=0)
    with pytest.raises(ValueError, match="weight holds"):
        zs.zs_layer_norm(out, F, 2, 8, 8, None, t[0, :7], None, F, 1e-5, None, out, 8, stream=0)
    with pytest.raises(ValueError, match="mean holds"):
        zs.zs_layer_norm(out, F, 2, 8, 8, None, None, None, F, 1e-5, None, out, 8,
                         torch.zeros(1), stream=0)
    with pytest.raises(ValueError, match="d_weight holds"):
        zs.zs_layer_norm_grad(out, out, F, 2, 8, 8, 8, None, F, t[0], t[0], None, t, out,
                              t[0, :7], None, F, stream=0)
    with pytest.raises(ValueError, match="one dtype"):
        zs.Tensors([t, t.bfloat16()])
    with pytest.raises(ValueError, match="contiguous"):
        zs.Tensors([t[:, :3]])
    with pytest.raises(ValueError, match="not dtype"):
        zs.zs_tensors_sqnorm([t], B, t, t, stream=0)
    with pytest.raises(ValueError, match="lengths"):
        zs.zs_tensors_scale([t], F, t, None, [t[:2]], F, stream=0)
    with pytest.raises(zs.ZsError):
        zs.zs_embedding_grad(out, F, 2, 8, 8, tok, 4, 1.0, None, torch.zeros(4), t, F, 8, stream=0)
