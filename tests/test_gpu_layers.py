"""The embedding lookup, layer norm and their gradients on the GPU against their
64-bit reference, within bounds derived from their roundings: widths 1 to 32768,
one row to thousands, every alignment and stride, padding, ids out of range, a
token repeated by the thousand, in place, offsets past 2^32, other streams,
captured and replayed."""
import math

import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import layers_reference as ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F, B = zs.ZS_FP32, zs.ZS_BF16
TYPE = ref.DTYPES
CANARY = 77.0


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Rows:
    """rows x dim of a dtype at any element offset and stride, with canaries
    between the rows and around them."""

    def __init__(self, rows, dim, dtype, pad=0, offset=0, values=None):
        self.rows, self.dim, self.stride = rows, dim, dim + pad
        self.buf = torch.full((offset + rows * self.stride + 16,), CANARY, dtype=TYPE[dtype],
                              device=DEV)
        flat = self.buf[offset:offset + rows * self.stride]
        self.view = flat.view(rows, self.stride)[:, :dim]
        self.address = self.view.data_ptr() if rows else self.buf[offset:].data_ptr()
        if values is not None:
            self.view.copy_(values)
        self.others = torch.ones_like(self.buf, dtype=torch.bool)
        self.others[offset:offset + rows * self.stride].view(rows, self.stride)[:, :dim] = False

    def untouched(self):
        return bool((self.buf[self.others] == CANARY).all())


def _normal(g, *shape, dtype=F, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(TYPE[dtype])


# ---------------------------------------------------------------- embedding ----
LOOKUPS = [  # rows, vocab, dim, table dtype, out dtype, pads, offsets, scale
    (1, 1, 1, B, B, 0, 0, 0, 0, 1.0), (1, 50257, 768, B, B, 0, 0, 0, 0, 1.0),
    (3, 5, 7, F, B, 0, 0, 0, 0, 2.5), (129, 1000, 256, B, F, 0, 0, 0, 0, 16.0),
    (64, 300, 1023, B, B, 0, 0, 0, 0, 0.5), (33, 100, 1025, F, F, 0, 1, 3, 1, -3.0),
    (17, 40, 2048, B, B, 8, 8, 8, 8, 45.25), (17, 40, 2048, B, B, 8, 0, 1, 0, 45.25),
    (17, 40, 2056, F, B, 4, 8, 4, 8, 1.0), (9, 64, 2049, B, F, 7, 3, 5, 2, 1e-3),
    (5, 3, 32768, B, B, 0, 0, 0, 0, 1.0), (1000, 32000, 4096, B, B, 0, 0, 0, 0, 64.0),
    (2, 4, 100, F, F, 28, 28, 0, 0, 0.0),
]


@pytest.mark.parametrize("case", LOOKUPS, ids=str)
def test_embedding(case):
    rows, vocab, dim, td, od, tpad, opad, toff, ooff, scale = case
    g = _gen(rows * 31 + dim)
    table = Rows(vocab, dim, td, tpad, toff, _normal(g, vocab, dim, dtype=td))
    out = Rows(rows, dim, od, opad, ooff)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    tokens[1::5] = -1
    zs.zs_embedding(table.address, td, vocab, dim, table.stride, tokens, rows, scale, out.address,
                    od, out.stride)
    want = ref.embedding(table.view.cpu(), tokens.cpu(), scale)
    ref.close(out.view, want, ref.tol_embedding(want, TYPE[od]), "out")
    assert out.untouched()
    if scale == 1.0 and td == od:
        assert torch.equal(out.view, torch.where(tokens[:, None] < 0, 0.0, table.view[tokens.clamp(min=0)]))


def test_embedding_ids_past_the_vocabulary():
    table, tokens = torch.ones(4, 8, device=DEV), torch.tensor([3, 4, -7, 1 << 40], device=DEV)
    out = torch.zeros(4, 8, device=DEV)
    zs.zs_embedding(table, F, 4, 8, 8, tokens, 4, 2.0, out, F, 8)
    with pytest.raises(zs.ZsError, match="token id") as e:
        zs.zs_check_device_error()
    assert e.value.status == zs.ZS_ERR_RANGE
    assert (out[0] == 2).all() and (out[2] == 0).all() and out[1].isnan().all() and out[3].isnan().all()
    d_table = torch.full((4, 8), CANARY, device=DEV)
    ws = torch.empty(zs.zs_embedding_grad_workspace_bytes(4, 8), dtype=torch.uint8, device=DEV)
    zs.zs_embedding_grad(table, F, 4, 8, 8, tokens, 4, 2.0, None, ws, d_table, F, 8)
    with pytest.raises(zs.ZsError, match="token id"):
        zs.zs_check_device_error()
    assert (d_table[:3] == 0).all() and (d_table[3] == 2).all()


def _tokens(g, rows, vocab, kind):
    if kind == "same":
        t = torch.full((rows,), vocab - 1, device=DEV)
    elif kind == "two":   # two long runs that meet inside a block
        t = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.41, 0, vocab - 1)
    elif kind == "zipf":
        u = torch.rand(rows, generator=g, device=DEV, dtype=torch.float64)
        t = ((vocab + 1.0) ** u).long().sub_(1).clamp_(0, vocab - 1)
    elif kind == "blocks":   # runs of 63, 64, 65, 96, 97, 31, 1, ... in scattered order
        lengths = torch.tensor([63, 64, 65, 96, 97, 31, 1, 33, 32, 128, 66, 2])
        t = torch.repeat_interleave(torch.arange(len(lengths)) % vocab, lengths)[:rows]
        t = torch.cat([t, torch.full((rows - len(t),), vocab - 1)]).to(DEV)
        t = t[torch.randperm(rows, generator=g, device=DEV)]
    elif kind == "none":
        t = torch.full((rows,), -1, device=DEV)
    else:
        t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        t[2::7] = -5
    return t.long()


GRADS = [  # rows, vocab, dim, d_out dtype, table dtype, pads, offsets, tokens, add
    (1, 1, 1, F, F, 0, 0, 0, 0, "any", None), (1, 1000, 256, B, B, 0, 0, 0, 0, "any", None),
    (31, 7, 64, B, F, 0, 0, 0, 0, "any", "other"), (32, 3, 65, F, B, 1, 0, 1, 1, "any", "self"),
    (33, 1, 255, F, F, 0, 0, 0, 0, "same", None), (65, 5, 256, B, B, 0, 0, 0, 0, "same", "self"),
    (64, 5, 257, B, F, 0, 0, 0, 0, "same", None), (512, 1000, 256, B, F, 0, 0, 0, 0, "any", None),
    (700, 12, 300, B, F, 4, 4, 0, 0, "blocks", "other"),
    (1000, 50, 512, F, F, 0, 8, 0, 4, "two", "self"),
    (4099, 50257, 96, B, F, 0, 0, 0, 0, "zipf", None),
    (4099, 50257, 96, B, B, 0, 0, 0, 0, "zipf", "self"),
    (3000, 1024, 768, B, B, 0, 0, 0, 0, "zipf", "other"),
    (5000, 1023, 130, F, F, 3, 5, 1, 2, "zipf", None),
    (100, 2, 32768, B, F, 0, 0, 0, 0, "two", None),
    (257, zs.ZS_MAX_VOCAB, 8, B, B, 0, 0, 0, 0, "any", None),
    (2100, 12, 300, B, F, 4, 4, 0, 0, "blocks", "other"),
    (2100, 12, 100, F, B, 0, 0, 0, 0, "blocks", "self"), (1025, 7, 40, F, F, 0, 0, 0, 0, "any", None),
    (1500, 5, 256, B, F, 0, 0, 0, 0, "same", "self"), (4000, 50, 65, F, F, 0, 0, 0, 0, "two", None),
    (1024, 3, 512, B, B, 0, 0, 0, 0, "same", "other"), (1024, 900, 8, B, F, 0, 0, 0, 0, "zipf", None),
    (3, zs.ZS_MAX_VOCAB, 8, F, B, 0, 0, 0, 0, "any", "self"),
    (40000, 3000, 64, F, F, 0, 0, 0, 0, "zipf", None), (40, 9, 16, F, F, 0, 0, 0, 0, "none", "other"),
    (0, 9, 16, F, B, 0, 0, 0, 0, "any", None), (0, 9, 16, F, B, 0, 0, 0, 0, "any", "other"),
    (0, 9, 16, F, B, 0, 0, 0, 0, "any", "self"),
]


@pytest.mark.parametrize("case", GRADS, ids=str)
def test_embedding_grad(case):
    rows, vocab, dim, od, td, dpad, tpad, doff, toff, kind, add = case
    g = _gen(rows * 17 + dim)
    tokens = _tokens(g, rows, vocab, kind)
    d = Rows(rows, dim, od, dpad, doff, _normal(g, rows, dim, dtype=od))
    scale = 1.75
    table = Rows(vocab, dim, td, tpad, toff)
    other = None
    base = _normal(g, vocab, dim, dtype=td) if add else None
    if add == "self":
        table.view.copy_(base)
    elif add:
        other = Rows(vocab, dim, td, tpad, toff, base)
    add_to = {None: None, "self": table.address, "other": other and other.address}[add]
    need = zs.zs_embedding_grad_workspace_bytes(rows, dim)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device=DEV)

    def call():
        zs.zs_embedding_grad(d.address, od, rows, dim, d.stride, tokens, vocab, scale, add_to,
                             ws[:need], table.address, td, table.stride)

    call()
    want, tol = ref.embedding_grad(d.view.cpu(), tokens.cpu(), vocab, scale,
                                   None if base is None else base.cpu())
    ref.close(table.view, want, tol + ref.rounding(want, TYPE[td]), "d_table")
    assert table.untouched() and d.untouched()
    assert (ws[need:] == 0xAB).all()
    if add == "self":   # rows without tokens keep their bits
        met = torch.zeros(vocab, dtype=torch.bool, device=DEV)
        met[tokens[tokens >= 0]] = True
        assert torch.equal(table.view[~met], base[~met])
    first = table.view.clone()
    if add == "self":
        table.view.copy_(base)
    call()
    assert torch.equal(first, table.view)   # the same bits again


def test_embedding_grad_sums_in_the_order_of_the_tokens():
    # 1e8 + 1 - 1e8 ...: what fp32 makes of this depends on the order
    rows = 15
    d = torch.tensor([1e8, 1.0, -1e8], device=DEV).repeat(rows // 3)[:, None].repeat(1, 4).contiguous()
    tokens = torch.full((rows,), 2, device=DEV)
    table = torch.empty(5, 4, device=DEV)
    ws = torch.empty(zs.zs_embedding_grad_workspace_bytes(rows, 4), dtype=torch.uint8, device=DEV)
    zs.zs_embedding_grad(d, F, rows, 4, 4, tokens, 5, 1.0, None, ws, table, F, 4)
    want = torch.zeros(4)
    for row in d.cpu():
        want = want + row
    assert torch.equal(table[2].cpu(), want)


def test_embedding_offsets_past_32_bits():
    far = (1 << 32) + 8
    table = torch.empty(far + 64, dtype=torch.bfloat16, device=DEV)
    table[:64] = 1.0
    table[far:] = 3.0
    tokens = torch.tensor([1, 0, 1], device=DEV)
    out = torch.empty(3, 64, dtype=torch.bfloat16, device=DEV)
    zs.zs_embedding(table, B, 2, 64, far, tokens, 3, 2.0, out, B, 64)
    assert out[:, 0].tolist() == [6.0, 2.0, 6.0] and out[:, 63].tolist() == [6.0, 2.0, 6.0]
    ws = torch.empty(zs.zs_embedding_grad_workspace_bytes(3, 64), dtype=torch.uint8, device=DEV)
    zs.zs_embedding_grad(out, B, 3, 64, 64, tokens, 2, 1.0, None, ws, table, B, far)
    assert (table[:64] == 2.0).all() and (table[far:] == 12.0).all()
    zs.zs_embedding_grad(table, B, 2, 64, far, tokens, 2, 1.0, None, ws, out, B, 64)
    assert (out[0] == 12.0).all() and (out[1] == 2.0).all()
    w = torch.empty(2, 64, dtype=torch.bfloat16, device=DEV)
    zs.zs_layer_norm(table, B, 2, 64, far, None, None, None, B, 1e-5, None, w, 64)
    assert (w == 0).all()


# --------------------------------------------------------------- layer norm ----
NORMS = [  # rows, dim, dtype, weight dtype, residual, weight, bias, pads (in, out), offset
    (1, 1, F, F, False, True, True, 0, 0, 0), (1, 768, B, B, True, True, True, 0, 0, 0),
    (2, 2, B, F, True, True, False, 0, 0, 0), (7, 33, F, B, False, False, False, 1, 0, 1),
    (128, 256, B, B, True, True, True, 0, 0, 0), (65, 767, B, F, True, True, True, 0, 0, 0),
    (65, 768, B, F, True, False, True, 8, 16, 8), (9, 1024, F, F, True, True, True, 0, 0, 0),
    (33, 1025, B, B, False, True, True, 3, 1, 1), (257, 2048, B, B, True, True, True, 0, 0, 0),
    (31, 4096, F, B, True, True, True, 4, 8, 0), (5, 4100, B, B, True, True, True, 0, 4, 2),
    (3, 8192, B, F, True, True, True, 0, 0, 0), (3, 8193, F, F, True, True, True, 0, 0, 0),
    (2, 16384, B, B, True, True, True, 0, 0, 0), (2, 32768, F, F, True, True, True, 0, 0, 0),
    (3, 32767, B, B, False, True, True, 0, 1, 1), (3001, 96, B, B, True, True, True, 0, 0, 0),
]


def _vector(g, dim, dtype, offset, sigma, mean=0.0):
    v = torch.full((dim + offset + 8,), CANARY, dtype=TYPE[dtype], device=DEV)
    v[offset:offset + dim] = (torch.randn(dim, generator=g, device=DEV) * sigma + mean).to(TYPE[dtype])
    return v[offset:offset + dim]


@pytest.mark.parametrize("case", NORMS, ids=str)
def test_layer_norm_and_its_gradient(case):
    rows, dim, dt, wd, residual, weight, bias, ipad, opad, offset = case
    g = _gen(rows * 13 + dim)
    T, eps = TYPE[dt], 1e-5
    loud = torch.where(torch.rand(dim, generator=g, device=DEV) < 0.02, 20.0, 1.0)
    x = Rows(rows, dim, dt, ipad, offset, _normal(g, rows, dim) * loud + 3.0)
    res = Rows(rows, dim, dt, ipad, offset, _normal(g, rows, dim)) if residual else None
    w = _vector(g, dim, wd, offset, 0.3, 1.0) if weight else None
    b = _vector(g, dim, wd, offset, 0.5) if bias else None
    total = Rows(rows, dim, dt, opad, offset) if residual else None
    y = Rows(rows, dim, dt, opad, offset)
    mean, rstd = torch.empty(2, rows, device=DEV)
    addr = lambda r: r and r.address  # noqa: E731
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    zs.zs_layer_norm(x.address, dt, rows, dim, x.stride, addr(res), ptr(w), ptr(b), wd, eps,
                     addr(total), y.address, y.stride, mean, rstd)
    h = x.view
    if residual:
        h = (x.view.float() + res.view.float()).to(T)
        assert torch.equal(total.view, h) and total.untouched()
    host = lambda t: None if t is None else t.cpu()  # noqa: E731
    want = ref.layer_norm(h.cpu(), host(w), host(b), eps)
    ref.close(y.view, want["y"], want["t_y"] + ref.rounding(want["y"], T), "y")
    ref.close(mean, want["mean"], want["t_mean"], "mean")
    ref.close(rstd, want["rstd"], want["t_rstd"], "rstd")
    assert y.untouched() and x.untouched()

    # the backward pass of the same rows, from these statistics
    hx = total if residual else x
    dy = Rows(rows, dim, dt, ipad, offset, _normal(g, rows, dim, sigma=0.1))
    past = Rows(rows, dim, dt, ipad, offset, _normal(g, rows, dim, sigma=0.1)) if residual else None
    dx = Rows(rows, dim, dt, ipad, offset)
    gd = F if wd == B else B
    dw, db = (torch.full((dim + 9,), CANARY, dtype=TYPE[gd], device=DEV) for _ in range(2))
    need = zs.zs_layer_norm_grad_workspace_bytes(rows, dim)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    want = ref.layer_norm_grad(dy.view.cpu(), h.cpu(), host(w), mean.cpu(), rstd.cpu(),
                               None if past is None else past.view.cpu())

    def call(to, dw, db):
        zs.zs_layer_norm_grad(dy.address, hx.address, dt, rows, dim, dy.stride, hx.stride, ptr(w),
                              wd, mean, rstd, addr(past), ws[:need], to, dw and dw.data_ptr(),
                              db and db.data_ptr(), gd)

    class At:
        def __init__(self, t):
            self.t = t

        def data_ptr(self):
            return self.t.data_ptr()

    call(dx.address, At(dw[1:]), At(db[1:]))
    ref.close(dx.view, want["d_x"], want["t_d_x"] + ref.rounding(want["d_x"], T), "d_x")
    for name, got in (("d_weight", dw), ("d_bias", db)):
        ref.close(got[1:1 + dim], want[name], want["t_" + name] + ref.rounding(want[name], TYPE[gd]), name)
        assert got[0] == CANARY and (got[1 + dim:] == CANARY).all()
    assert dx.untouched() and dy.untouched() and (ws[need:] == 0xAB).all()
    # one sum alone, then in place of the incoming gradient: the same bits
    one = torch.empty(dim, dtype=TYPE[gd], device=DEV)
    again = Rows(rows, dim, dt, ipad, offset)
    call(again.address, At(one), None)
    assert torch.equal(one, dw[1:1 + dim]) and torch.equal(again.view, dx.view)
    call(again.address, None, At(one))
    assert torch.equal(one, db[1:1 + dim])
    call(dy.address, None, None)
    assert torch.equal(dy.view, dx.view) and dy.untouched()


@pytest.mark.parametrize("dim", [64, 768, 4096])
def test_layer_norm_in_place(dim):
    g = _gen(dim)
    rows = 37
    x, res = (_normal(g, rows, dim, dtype=B) for _ in range(2))
    w = _normal(g, dim, dtype=B)
    total, y = torch.empty_like(x), torch.empty_like(x)

    def call(x, res, total, y):
        zs.zs_layer_norm(x, B, rows, dim, dim, res, w, None, B, 1e-5, total, y, dim)

    call(x, res, total, y)
    a, r = x.clone(), res.clone()
    call(a, r, r, a)          # the stream takes the sum, the branch its norm
    assert torch.equal(a, y) and torch.equal(r, total)
    a, r = x.clone(), res.clone()
    call(a, r, a, r)
    assert torch.equal(a, total) and torch.equal(r, y)
    a = x.clone()
    call(a, res, None, a)
    assert torch.equal(a, y)


def test_layer_norm_hard_rows():
    dim, eps = 500, 1e-6
    base = torch.randn(dim, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    rows = torch.stack([
        torch.zeros(dim), torch.full((dim,), 5.0), torch.full((dim,), -300.0),   # no deviation
        base.float() * 1e-3 + 1000.0,        # deviations of a ten-thousandth of the mean
        base.float() * 1e-12, base.float() * 1e17, base.float(), base.float(), base.float()])
    rows[6, 17] = math.inf
    rows[7, 499] = math.nan
    x = rows.to(DEV)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(2, len(rows), device=DEV)
    zs.zs_layer_norm(x, F, len(rows), dim, dim, None, None, None, F, eps, None, y, dim, mean, rstd)
    want = ref.layer_norm(rows, None, None, eps)
    # an infinite row's values are not numbers, all of them
    assert y[6:8].isnan().all() and rstd[6:8].isnan().all() and mean[7].isnan()
    keep = [0, 1, 2, 3, 4, 5, 8]
    ref.close(y[keep], want["y"][keep], (want["t_y"] + ref.rounding(want["y"], torch.float32))[keep], "y")
    ref.close(mean[keep], want["mean"][keep], want["t_mean"][keep], "mean")
    ref.close(rstd[keep], want["rstd"][keep], want["t_rstd"][keep], "rstd")


def test_layer_norm_grad_of_many_rows_and_of_none():
    g = _gen(5)
    rows, dim = 9001, 72
    x, dy = (_normal(g, rows, dim) for _ in range(2))
    st = ref.layer_norm(x.cpu(), None, None, 1e-5)
    mean, rstd = (st[k].float().to(DEV) for k in ("mean", "rstd"))
    ws = torch.empty(zs.zs_layer_norm_grad_workspace_bytes(rows, dim), dtype=torch.uint8, device=DEV)
    dx, dw, db = torch.empty_like(x), *torch.empty(2, dim, device=DEV)
    zs.zs_layer_norm_grad(dy, x, F, rows, dim, dim, dim, None, F, mean, rstd, None, ws, dx, dw, db, F)
    want = ref.layer_norm_grad(dy.cpu(), x.cpu(), None, mean.cpu(), rstd.cpu(), None)
    for name, got in (("d_x", dx), ("d_weight", dw), ("d_bias", db)):
        ref.close(got, want[name], want["t_" + name] + ref.rounding(want[name], torch.float32), name)
    zs.zs_layer_norm_grad(None, None, F, 0, dim, dim, dim, None, F, None, None, None, None, None,
                          dw, db, F)
    assert (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------- streams and graphs ----
def _step_buffers(g, rows=200, vocab=97, dim=192):
    s = dict(rows=rows, vocab=vocab, dim=dim)
    s["table"] = _normal(g, vocab, dim, dtype=B)
    s["tokens"] = torch.randint(-1, vocab, (rows,), generator=g, device=DEV)
    s["w"], s["b"] = _normal(g, dim, dtype=B), _normal(g, dim, dtype=B)
    s["dy"] = _normal(g, rows, dim, dtype=B)
    for name in ("e", "h", "y", "dx"):
        s[name] = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    s["mean"], s["rstd"] = torch.zeros(2, rows, device=DEV)
    s["dw"], s["db"] = torch.zeros(2, dim, device=DEV)
    s["dt"] = torch.zeros(vocab, dim, device=DEV)
    s["ws"] = torch.empty(max(zs.zs_embedding_grad_workspace_bytes(rows, dim),
                              zs.zs_layer_norm_grad_workspace_bytes(rows, dim)),
                          dtype=torch.uint8, device=DEV)
    return s


def _step(s, stream=None):
    R, V, D = s["rows"], s["vocab"], s["dim"]
    zs.zs_embedding(s["table"], B, V, D, D, s["tokens"], R, 2.0, s["e"], B, D, stream=stream)
    zs.zs_layer_norm(s["e"], B, R, D, D, s["dy"], s["w"], s["b"], B, 1e-5, s["h"], s["y"], D,
                     s["mean"], s["rstd"], stream=stream)
    zs.zs_layer_norm_grad(s["dy"], s["h"], B, R, D, D, D, s["w"], B, s["mean"], s["rstd"], s["y"],
                          s["ws"], s["dx"], s["dw"], s["db"], F, stream=stream)
    zs.zs_embedding_grad(s["dx"], B, R, D, D, s["tokens"], V, 2.0, None, s["ws"], s["dt"], F, D,
                         stream=stream)
    return [s[k] for k in ("e", "h", "y", "mean", "rstd", "dx", "dw", "db", "dt")]


@pytest.mark.parametrize("rows,dim", [(200, 192), (3000, 192), (70, 8200)])
def test_another_stream_and_a_graph_give_the_same_bits(rows, dim):
    s = _step_buffers(_gen(9), rows, 97, dim)
    want = [t.clone() for t in _step(s)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for t in _step(s):
        t.zero_()
    torch.cuda.synchronize()
    got = _step(s, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured; replayed on other inputs in the same buffers
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(s)
    other = _step_buffers(_gen(10), rows, 97, dim)
    want = [t.clone() for t in _step(other)]
    for name in ("table", "tokens", "w", "b", "dy"):
        s[name].copy_(other[name])
    for _ in range(3):
        for t in got:
            t.fill_(CANARY)
        s["ws"].fill_(0xCD)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_that_share_a_workspace():
    a, b = _step_buffers(_gen(11), rows=2500), _step_buffers(_gen(12), rows=1333, vocab=31, dim=96)
    want = [[t.clone() for t in _step(s)] for s in (a, b)]
    big = max(a["ws"], b["ws"], key=len)
    a["ws"] = b["ws"] = big
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            _step(s)
    for order in ((0, 1), (1, 0), (0, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        names = ("e", "h", "y", "mean", "rstd", "dx", "dw", "db", "dt")
        for i in set(order):
            s = (a, b)[i]
            assert all(torch.equal(s[k], w) for k, w in zip(names, want[i]))


def test_many_threads_at_once():
    """Eight host threads, each on its own stream and buffers, widths whose kernels
    ask for different amounts of shared memory: each gets what it gets alone."""
    import threading
    shapes = [(300, 97, 768), (2000, 31, 768), (40, 9, 4096), (700, 97, 2048), (5, 9, 8192),
              (900, 50, 768), (1500, 31, 2048), (64, 9, 1000)]
    sets = [_step_buffers(_gen(20 + i), *x) for i, x in enumerate(shapes)]
    want = [[t.clone() for t in _step(s)] for s in sets]
    torch.cuda.synchronize()
    streams, wrong = [torch.cuda.Stream() for _ in sets], []

    def work(i):
        for _ in range(30):
            got = _step(sets[i], stream=streams[i])
        streams[i].synchronize()
        if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


@pytest.mark.parametrize("overlap", [1, 0])
@pytest.mark.parametrize("rows,dim,td", [(3000, 256, F), (2500, 768, B), (200, 320, F)])
def test_dependent_calls_back_to_back(rows, dim, td, overlap):
    """Gradients of other tokens into one table, one after another without a wait,
    each added to the one before or starting anew, and each read by a lookup that
    follows: as when every call is waited for."""
    g, vocab, n = _gen(rows), 700, 12
    tokens = [_tokens(g, rows, vocab, "zipf") for _ in range(n)]
    d = [_normal(g, rows, dim, dtype=B) for _ in range(n)]
    ws = torch.empty(zs.zs_embedding_grad_workspace_bytes(rows, dim), dtype=torch.uint8, device=DEV)
    all_rows = torch.arange(vocab, device=DEV)

    def chain(wait):
        a, b = torch.zeros(2, vocab, dim, dtype=TYPE[td], device=DEV)
        outs = []
        for i in range(n):
            base = {0: None, 1: a, 2: b}[i % 3]   # anew, in place, added to another
            zs.zs_embedding_grad(d[i], B, rows, dim, dim, tokens[i], vocab, 1.5, base, ws, a, td, dim)
            if wait:
                torch.cuda.synchronize()
            out = torch.empty(vocab, dim, dtype=TYPE[td], device=DEV)
            zs.zs_embedding(a, td, vocab, dim, dim, all_rows, vocab, 1.0, out, td, dim)
            outs.append(out)
            if i % 3 == 0:
                b.copy_(a)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    old = zs.zs_set_launch_overlap(overlap)
    try:
        want, got = chain(True), chain(False)
    finally:
        zs.zs_set_launch_overlap(old)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_launch_overlap_changes_no_bits():
    s = _step_buffers(_gen(40), rows=2100, vocab=61, dim=768)
    want = [t.clone() for t in _step(s)]
    old = zs.zs_set_launch_overlap(0)
    try:
        got = _step(s)
        torch.cuda.synchronize()
    finally:
        zs.zs_set_launch_overlap(old)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
