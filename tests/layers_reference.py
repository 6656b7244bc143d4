"""The operators around the layers in 64 bits, from their definitions, and the
error bounds the kernels are held to.

Bounds (eps = 2^-24, one fp32 rounding; first order). A row's sums are chains of
at most 32 elements of a lane, 5 steps between lanes and 32 warps: 70 additions.
A rounding of the result to bf16 is off by at most 2^-8 of it."""
import torch

EPS = 2.0 ** -24
BF16_ROUNDING = 2.0 ** -8
TINY = 2.0 ** -126      # a result below it may lose digits or be flushed
CHAIN = 70
DTYPES = {0: torch.bfloat16, 1: torch.float32}   # by zs dtype


def rounding(ref, dtype):
    return ref.abs() * (BF16_ROUNDING if dtype == torch.bfloat16 else EPS) + TINY


def embedding(table, tokens, scale):
    """float64 rows; NaN for ids past the vocabulary, 0 for negative ones."""
    V = table.shape[0]
    rows = table.double()[tokens.clamp(0, V - 1)] * scale
    rows[tokens < 0] = 0.0
    rows[tokens >= V] = float("nan")
    return rows


def tol_embedding(ref, dtype):
    """The scale rounded to fp32, the product, the result."""
    return 2 * EPS * ref.abs() + rounding(ref, dtype)


def embedding_grad(d_out, tokens, vocab, scale, add):
    """(gradient, its tolerance before the last rounding)."""
    some = (tokens >= 0) & (tokens < vocab)
    at = tokens[some]
    d = d_out.double()[some]
    ref, size, n = (torch.zeros(vocab, d_out.shape[1], dtype=torch.float64) for _ in range(3))
    ref.index_add_(0, at, d)
    size.index_add_(0, at, d.abs())
    n.index_add_(0, at, torch.ones_like(d))
    # a run's sum: no more additions than terms; then the scale, and the sum with add
    tol = (n + 3) * EPS * size * abs(scale)
    ref = ref * scale
    if add is not None:
        tol = tol + EPS * (add.double().abs() + ref.abs())
        ref = ref + add.double()
    return ref, tol


def layer_norm(h, weight, bias, eps):
    """dict of y, mean, rstd and their tolerances (before y's last rounding)."""
    h = h.double()
    mean = h.mean(1, keepdim=True)
    d = h - mean
    rstd = (d.square().mean(1, keepdim=True) + eps) ** -0.5
    w = torch.ones(h.shape[1], dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    xh = d * rstd
    y = xh * w + b
    spread = d.abs().mean(1, keepdim=True)
    # deviations are rounded once, their mean is a chain of them and corrects the
    # first mean, which is off by a chain of its own (second order, but of the mean)
    first = CHAIN * EPS * mean.abs()
    t_d = EPS * (3 * d.abs() + (CHAIN + 4) * spread) + CHAIN * EPS * first
    # var is a chain of squares less that correction's square, its root halves both
    t_rstd = EPS * (CHAIN / 2 + 8) * rstd + CHAIN * EPS * first.square() * rstd ** 3
    t_y = w.abs() * (rstd * t_d + t_rstd * d.abs()) + EPS * (4 * (xh * w).abs() + 2 * b.abs())
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], t_y=t_y,
                t_mean=(EPS * (2 * mean.abs() + (CHAIN + 4) * spread) + CHAIN * EPS * first)[:, 0] + TINY,
                t_rstd=t_rstd[:, 0])


def layer_norm_grad(dy, x, weight, mean, rstd, d_sum):
    """dict of d_x, d_weight, d_bias and their tolerances before the last
    rounding, from the given statistics."""
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    R, D = x.shape
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double()
    xh = (x - mean) * rstd           # two roundings
    g = dy * w                       # one
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    t_dx = rstd * EPS * (5 * g.abs() + (CHAIN + 8) * (a1 + xh.abs() * a2) + 8 * (xh * c2).abs())
    if d_sum is not None:
        dx = dx + d_sum.double()
        t_dx = t_dx + EPS * (d_sum.double().abs() + dx.abs())
    # a group's rows, 8 groups of a block, then the blocks in two chains
    chain = R / 304 + 2 + 8 + 304 / 8 + 8
    return dict(d_x=dx, t_d_x=t_dx,
                d_weight=(dy * xh).sum(0), t_d_weight=EPS * (chain + 3) * (dy * xh).abs().sum(0),
                d_bias=dy.sum(0), t_d_bias=EPS * chain * dy.abs().sum(0))


def sqnorm(tensors):
    return sum(float(t.double().square().sum()) for t in tensors)


T_SQNORM = 9 * EPS   # chains of eight squares at most, joined twice, in fp32; then double


def close(got, ref, tol, what):
    """|got - ref| <= tol elementwise; NaN with NaN, infinities equal."""
    got = got.double().cpu()
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} against {tuple(ref.shape)}"
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN pattern"
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~ref.isnan()], ref[~fine & ~ref.isnan()]), f"{what}: infinities"
    off = (got - ref).abs()[fine] - torch.as_tensor(tol).expand_as(ref)[fine]
    assert off.numel() == 0 or off.max() <= 0, \
        f"{what}: {int((off > 0).sum())} of {off.numel()} past the bound, by {float(off.max()):.3g}"
