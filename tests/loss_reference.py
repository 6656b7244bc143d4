"""The vocabulary-row losses in 64 bits, from their definitions, and the error
bounds the fp32 kernels are held to.

Bounds (eps = 2^-24, one fp32 rounding). With d = (z - M)/T and e = exp(d):
three roundings act on d and the exponential is good to 4 eps, so e is off by
at most (3 |d| + 4) eps, which averages to at most (3 ln V + 4) eps over S =
sum e (sum p |d| <= ln V). A sum of V terms whose longest chain of additions
has V/256 + 64 links adds that many eps. The other bounds follow from the
formulas, first order, one eps per further operation."""
import math

import torch

EPS = 2.0 ** -24
BF16_ROUNDING = 2.0 ** -8   # 8 significant bits: half a unit in the last place
TINY = 1e-36   # results below it may be flushed to zero


def _masked_log_softmax(y):
    """(ln p, lse) with lse = -inf and ln p = -inf for a row masked throughout."""
    m = y.amax(1, keepdim=True)
    m0 = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
    d = y - m0   # formed first: for a row of the type's lowest value, m + ln s rounds to m
    ln_s = d.exp().sum(1, keepdim=True).log()
    lse = m0 + ln_s
    lnp = torch.where(torch.isneginf(ln_s), torch.full_like(y, -math.inf), d - ln_s)
    return lnp, lse[:, 0]


def _pick(lnp, targets):
    V = lnp.shape[1]
    some = (targets >= 0) & (targets < V)
    x = lnp.gather(1, torch.where(some, targets, 0)[:, None])[:, 0]
    return torch.where(targets >= V, torch.full_like(x, math.nan),
                       torch.where(some, x, torch.zeros_like(x)))


def token_logprobs(z, targets, T):
    """dict of logprob, entropy, lse for float64 logits z [R, V]."""
    lnp, lse = _masked_log_softmax(z / T)
    p = lnp.exp()
    ent = -torch.where(p == 0, torch.zeros_like(p), p * lnp).sum(1)
    out = dict(entropy=ent, lse=lse, lnp=lnp)
    if targets is not None:
        out["logprob"] = _pick(lnp, targets)
    return out


def top(z, k):
    """Ids of the k largest, equal values lowest id first, NaN above all."""
    key = torch.where(torch.isnan(z), torch.full_like(z, math.inf), z)
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    nan = torch.isnan(z).gather(1, order)
    order = order.gather(1, torch.argsort((~nan).int(), dim=1, stable=True))
    return order[:, :k]


def teacher(ids, t, teacher_lse, T, V):
    """q, ln q and usable ids [R, K] (q = 0 at unused entries)."""
    used = (ids >= 0) & (ids < V)
    u = torch.where(used, t / T, torch.full_like(t, -math.inf))
    if teacher_lse is None:
        lnq, _ = _masked_log_softmax(u)
    else:
        lnq = u - teacher_lse[:, None]
    q = torch.where(used, lnq.exp(), torch.zeros_like(lnq))
    return q, torch.where(q == 0, torch.zeros_like(lnq), lnq), torch.where(used, ids, 0).long()


def distill(z, ids, t, teacher_lse, T, targets):
    out = {}
    lnp, out["lse"] = _masked_log_softmax(z / T)
    if ids is not None:
        q, lnq, at = teacher(ids, t, teacher_lse, T, z.shape[1])
        out["loss"] = torch.where(q == 0, torch.zeros_like(q), q * (lnq - lnp.gather(1, at))).sum(1)
    ln1, out["hard_lse"] = _masked_log_softmax(z)
    if targets is not None:
        out["logprob"] = _pick(ln1, targets)
    return out


def _weights(x, R):
    return torch.zeros(R, dtype=torch.float64) if x is None else x.double()


def token_grad(z, targets, T, lse, entropy, d_logprob, d_entropy):
    """The gradient from the given normalisers (fp32 values of the forward call)."""
    R, V = z.shape
    a, b = _weights(d_logprob, R), _weights(d_entropy, R)
    if targets is not None:
        a = torch.where((targets >= 0) & (targets < V), a, 0.0)
    lnp = z / T - lse.double()[:, None]
    p = lnp.exp()
    H = torch.zeros(R, dtype=torch.float64) if entropy is None else entropy.double()
    ent = torch.where(p == 0, torch.zeros_like(p), p * (lnp + H[:, None]))
    g = -a[:, None] * p - b[:, None] * ent
    if targets is not None:
        g.scatter_add_(1, targets.clamp(0, V - 1)[:, None], a[:, None])
    off = torch.isneginf(lse) | ((a == 0) & (b == 0))
    return torch.where(off[:, None], 0.0, g / T)


def distill_grad(z, ids, t, teacher_lse, T, targets, lse, hard_lse, d_loss, d_logprob):
    R, V = z.shape
    w, h = _weights(d_loss, R), _weights(d_logprob, R)
    if targets is not None:
        h = torch.where((targets >= 0) & (targets < V), h, 0.0)
    g = torch.zeros_like(z)
    off = (w == 0) & (h == 0)
    if d_loss is not None:
        q, _, at = teacher(ids, t, teacher_lse, T, V)
        p = (z / T - lse.double()[:, None]).exp()
        g += (w / T * q.sum(1))[:, None] * p
        g.scatter_add_(1, at, -(w / T)[:, None] * q)
        off = off | torch.isneginf(lse)
    if d_logprob is not None:
        g -= h[:, None] * (z - hard_lse.double()[:, None]).exp()
        g.scatter_add_(1, targets.clamp(0, V - 1)[:, None], h[:, None])
        off = off | torch.isneginf(hard_lse)
    return torch.where(off[:, None], 0.0, g)


# ----------------------------------------------------------------- bounds ----
def _finite_abs(x):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))


def tol_sum(V):
    """Relative error of S."""
    return EPS * (3 * math.log(V) + 4 + V / 256 + 64)


def tol_lse(z, lse, T):
    M = _finite_abs(z.amax(1) / T)
    return tol_sum(z.shape[1]) + 4 * EPS * (M + _finite_abs(lse))


def tol_logprob(z, logprob, T, V):
    """ln p = (z - M)/T - ln S, |z - M|/T <= |ln p| + ln V."""
    return tol_sum(V) + 4 * EPS * (2 * _finite_abs(logprob) + 2 * math.log(V) + 1)


def tol_entropy(V):
    return tol_sum(V) * (1 + 2 * (math.log(V) + 1)) + 4 * EPS * (math.log(V) + 1)


def tol_q(t, T, teacher_lse):
    """Absolute error of ln q, relative of q, per row."""
    big = _finite_abs(t / T).amax(1)
    if teacher_lse is not None:
        big = big + _finite_abs(teacher_lse.double())
    return EPS * (4 * big + 64)


def tol_loss(z, ids, t, teacher_lse, T, lnp_at, q, lnq):
    V = z.shape[1]
    tq = tol_q(t, T, teacher_lse)[:, None]
    term = _finite_abs(lnq - lnp_at)
    each = tq * (1 + term) + tol_logprob(z, lnp_at, T, V) + 16 * EPS * term
    return (q * each).sum(1) + EPS


def tol_grad(z, T, lse, coef, V, bf16, g, special):
    """|g - ref|: coef [R] multiplies p (and p times its logarithm's size), the
    special columns add `special` [R]; a bf16 result rounds once more."""
    lse = lse.double()[:, None]
    y = z / T
    p = torch.where(torch.isneginf(lse), torch.zeros_like(y), (y - lse).exp())
    size = torch.where(p > 0, y.abs(), torch.zeros_like(y)) + _finite_abs(lse)
    tol = coef[:, None] * p * (tol_sum(V) + EPS * (8 * size + 32)) + special[:, None]
    tol = tol + 4 * EPS * g.abs() + TINY
    return tol + g.abs() * BF16_ROUNDING if bf16 else tol
