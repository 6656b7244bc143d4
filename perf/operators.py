"""What the vocabulary-row operators are measured on: log probabilities of
given tokens (with entropy and top alternatives) and distillation from a
teacher's top logits, each with its gradient.

Vocabularies are those of the repository's parameter lists (1000, 32000, 50257,
151936); rows are tokens of a batch. ``op`` names the call of a case:
  logprobs           zs_token_logprobs
  logprobs_grad      zs_token_logprobs_grad
  distill            zs_distill_loss
  distill_grad       zs_distill_grad
  distill_loss_grad  zs_distill_loss_grad
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
MOST_ELEMENTS = 8192 * 151936   # the largest listed case
MOST_RANKED = 8191 * 32000      # with top alternatives (the plain form ranks 64-bit keys)
IGNORED = 1.0 / 16              # share of rows with no target and no weight


def _case(name, op, rows, vocab, dtype, pad=0, top_k=0, teacher_k=0, teacher="fp32",
          teacher_lse=False, hard=False, entropy=True, temperature=1.0, mask="none"):
    return dict(name=name, op=op, rows=rows, vocab=vocab, dtype=dtype, pad=pad, top_k=top_k,
                teacher_k=teacher_k, teacher=teacher, teacher_lse=teacher_lse, hard=hard,
                entropy=entropy, temperature=temperature, mask=mask)


def listed():
    return [
        # One sampled token's log probability and five alternatives: a serving step, all latency.
        _case("logprobs one token", "logprobs", 1, 50257, "bf16", top_k=5),
        # A decoding batch that reports 20 alternatives at its sampling temperature; the
        # vocabulary's unused tail is masked out.
        _case("logprobs decode batch", "logprobs", 64, 151936, "bf16", top_k=20, temperature=0.7,
              mask="inf"),
        # Scoring a batch of sequences (4 x 1024 tokens) under the policy.
        _case("logprobs score", "logprobs", 4096, 151936, "bf16"),
        # A teacher's pass that records its 64 top tokens for a student, fp32 logits.
        _case("logprobs teacher record", "logprobs", 8191, 32000, "fp32", top_k=64),
        # The tiny model's eight tokens.
        _case("logprobs_grad tiny", "logprobs_grad", 8, 1000, "bf16"),
        # A policy-gradient step with an entropy bonus at an odd vocabulary (rows of every
        # alignment).
        _case("logprobs_grad policy", "logprobs_grad", 8192, 50257, "bf16"),
        # Evaluating a student on a few tokens; the teacher's own normaliser is recorded.
        _case("distill few tokens", "distill", 7, 50257, "fp32", teacher_k=20, teacher_lse=True),
        # Evaluating a student on a batch, soft and hard loss.
        _case("distill evaluate", "distill", 8192, 32000, "bf16", teacher_k=64, teacher="bf16",
              hard=True, temperature=2.0),
        # The gradient alone, logits and gradient in a buffer of padded rows.
        _case("distill_grad padded rows", "distill_grad", 1023, 50257, "fp32", pad=47,
              teacher_k=32, teacher_lse=True),
        # A training step of the tiny model: loss and gradient of 128 tokens.
        _case("distill_loss_grad tiny", "distill_loss_grad", 128, 1000, "bf16", teacher_k=16,
              hard=True),
        # A training step, hard labels mixed in at T = 1.
        _case("distill_loss_grad step", "distill_loss_grad", 4095, 32000, "bf16", teacher_k=64,
              hard=True, mask="lowest"),
        # The largest: a training step over 8192 tokens of the largest vocabulary.
        _case("distill_loss_grad large", "distill_loss_grad", 8192, 151936, "bf16", teacher_k=128,
              teacher="bf16", hard=True, temperature=2.0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "distill", "distill_grad", "distill_loss_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    vocab = _log_uniform(rng, 1000, 151936)
    top_k = _log_uniform(rng, 1, 128) if op == "logprobs" and rng.random() < 0.6 else 0
    most = (MOST_RANKED if top_k else MOST_ELEMENTS) // (BYTES[dtype] // 2)
    rows = _log_uniform(rng, 1, min(16384, most // vocab))
    distill = op.startswith("distill")
    return dict(op=op, rows=rows, vocab=vocab, dtype=dtype,
                pad=rng.choice([0, 0, 1, 64 - vocab % 64]), top_k=top_k,
                teacher_k=_log_uniform(rng, 1, 256) if distill else 0,
                teacher=rng.choice(["bf16", "fp32"]), teacher_lse=rng.random() < 0.5,
                hard=distill and rng.random() < 0.6, entropy=distill or rng.random() < 0.7,
                temperature=rng.choice([1.0, 1.0, 2.0, round(rng.uniform(0.5, 4.0), 3)]),
                mask=rng.choice(["none", "inf", "lowest"]))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["rows"] * 7 + case["vocab"])
    R, V, K = case["rows"], case["vocab"], case["teacher_k"]
    ld, T, dt = V + case["pad"], case["temperature"], DTYPES[case["dtype"]]
    f32 = dict(dtype=torch.float32, device=dev)

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, sigma, generator=g)

    buf = normal(R, ld, sigma=2.5, dtype=dt)
    logits = buf[:, :V]
    # the token the model is sure of, to a varying degree
    live = V if case["mask"] == "none" else V - V // 100
    targets = torch.randint(0, live, (R,), generator=g, device=dev)
    logits.scatter_(1, targets[:, None], (normal(R, 1).abs() * 6 + 4).to(dt))
    ignored = torch.rand(R, generator=g, device=dev) < IGNORED
    keep = (~ignored).float()
    s = dict(case=case, logits=buf, R=R, V=V, ld=ld, T=T)
    if K:
        # the teacher's K tokens (distinct in a row, the likely one first) and its logits for them
        step = torch.randint(1, live // K + 1, (R, 1), generator=g, device=dev)
        start = torch.where(ignored[:, None], torch.zeros_like(step), targets[:, None])
        ids = (start + step * torch.arange(K, device=dev)) % live
        t = torch.sort(normal(R, K, sigma=2.0) + 4.0, dim=1, descending=True).values
        logits.scatter_(1, ids, (t + 0.7 * normal(R, K)).to(dt))
        s["teacher_logits"] = t.to(DTYPES[case["teacher"]])
        # every eighth row's record is shorter than K
        short = torch.arange(R, device=dev) % 8 == 7
        ids[short, K - K // 4:] = -1
        s["teacher_ids"] = ids.to(torch.int32)
        s["teacher_lse"] = None
        if case["teacher_lse"]:
            rest = 1.0 + torch.rand(R, 1, generator=g, device=dev)
            s["teacher_lse"] = (torch.logsumexp(s["teacher_logits"].double() / T, 1)
                                + 0.1 * rest[:, 0].double()).float()
    if case["mask"] != "none":
        # the vocabulary's unused tail
        low = -math.inf if case["mask"] == "inf" else torch.finfo(dt).min
        logits[:, live:] = low
    s["targets"] = None
    if not K or case["hard"]:
        s["targets"] = torch.where(ignored, torch.full_like(targets, -100), targets)
    out = dict(logprob=torch.empty(R, **f32), entropy=torch.empty(R, **f32),
               lse=torch.empty(R, **f32), loss=torch.empty(R, **f32),
               hard_lse=torch.empty(R, **f32))
    if case["op"] == "logprobs" and case["top_k"]:
        out["top_ids"] = torch.empty(R, case["top_k"], dtype=torch.int32, device=dev)
        out["top_logprobs"] = torch.empty(R, case["top_k"], **f32)
    if case["op"].endswith("grad"):
        out["d_logits"] = torch.empty(R, ld, dtype=dt, device=dev)
        s["d_loss"] = keep * (0.5 + torch.rand(R, generator=g, device=dev)) / R
        s["d_logprob"] = -keep * (0.5 + torch.rand(R, generator=g, device=dev)) / R
        s["d_entropy"] = keep * normal(R) * 0.1 / R if case["entropy"] else None
    if case["op"] in ("logprobs_grad", "distill_grad"):
        # what the forward pass left
        s["lse"], s["entropy"], s["hard_lse"] = (torch.empty(R, **f32) for _ in range(3))
        for i in range(0, R, 512):
            z = logits[i:i + 512].double()
            logp = torch.log_softmax(z / T, 1)
            s["lse"][i:i + 512] = torch.logsumexp(z / T, 1)
            s["entropy"][i:i + 512] = -torch.where(logp > -700, logp.exp() * logp, 0.0).sum(1)
            s["hard_lse"][i:i + 512] = torch.logsumexp(z, 1)
    s["out"] = out
    return s


def _returned(case):
    """The names of the outputs of a case."""
    if case["op"] == "logprobs":
        return ["logprob", "entropy", "lse"] + (["top_ids", "top_logprobs"] if case["top_k"] else [])
    if case["op"] == "logprobs_grad" or case["op"] == "distill_grad":
        return ["d_logits"]
    names = ["loss", "lse"] + (["logprob", "hard_lse"] if case["hard"] else [])
    return names + (["d_logits"] if case["op"] == "distill_loss_grad" else [])


def _run_own(s):
    import fsdp_sharded_mixed_gb300 as zs
    case, o = s["case"], s["out"]
    code = zs.ZS_BF16 if case["dtype"] == "bf16" else zs.ZS_FP32
    rows = (s["logits"], code, s["R"], s["V"], s["ld"])
    op, T, hard = case["op"], s["T"], case["hard"]
    if op == "logprobs":
        zs.zs_token_logprobs(*rows, s["targets"], T, o["logprob"], o["entropy"], o["lse"],
                             case["top_k"], o.get("top_ids"), o.get("top_logprobs"))
    elif op == "logprobs_grad":
        zs.zs_token_logprobs_grad(*rows, s["targets"], T, s["lse"], s["entropy"], s["d_logprob"],
                                  s["d_entropy"], o["d_logits"], s["ld"])
    else:
        teacher = (s["teacher_ids"], s["teacher_logits"],
                   zs.ZS_BF16 if case["teacher"] == "bf16" else zs.ZS_FP32, case["teacher_k"],
                   s["teacher_lse"])
        logprob, hard_lse = (o["logprob"], o["hard_lse"]) if hard else (None, None)
        d_logprob = s["d_logprob"] if hard and op != "distill" else None
        if op == "distill":
            zs.zs_distill_loss(*rows, *teacher, T, s["targets"], o["loss"], o["lse"], logprob,
                               hard_lse)
        elif op == "distill_grad":
            zs.zs_distill_grad(*rows, *teacher, T, s["targets"], s["lse"],
                               s["hard_lse"] if hard else None, s["d_loss"], d_logprob,
                               o["d_logits"], s["ld"])
        else:
            zs.zs_distill_loss_grad(*rows, *teacher, T, s["targets"], s["d_loss"], d_logprob,
                                    o["loss"], o["lse"], logprob, hard_lse, o["d_logits"],
                                    s["ld"])
    got = {name: o[name] for name in _returned(case)}
    if "d_logits" in got:
        got["d_logits"] = got["d_logits"][:, :s["V"]]
    return got


def _plain_softmax(z, T):
    """(y - max, sum of exp, lse) of y = z / T in 32 bits."""
    y = z / T
    m = y.amax(1, keepdim=True)
    d = y - m
    total = d.exp().sum(1, keepdim=True)
    return d, total, (m + total.log())[:, 0]


def _plain_top(z, k):
    """The k largest, ties to the lowest index: 64-bit keys of value and index."""
    bits = (z + 0.0).contiguous().view(torch.int32)
    ordered = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    V = z.shape[1]
    back = torch.arange(V - 1, -1, -1, device=z.device)
    keys = torch.topk(ordered * (1 << 32) + back, k, dim=1, sorted=True).values
    return V - 1 - (keys & 0xFFFFFFFF)


def _plain_teacher(s):
    """q and ln q of the teacher's record (0 and 0 where it has no entry), and the ids."""
    ids = s["teacher_ids"].long()
    valid = ids >= 0
    u = torch.where(valid, s["teacher_logits"].float() / s["T"], -math.inf)
    if s["teacher_lse"] is None:
        u = u - u.amax(1, keepdim=True)
        logq = u - u.exp().sum(1, keepdim=True).log()
    else:
        logq = u - s["teacher_lse"][:, None]
    q = logq.exp()
    return q, torch.where(valid, logq, 0.0), ids.clamp(min=0)


def _run_plain(s):
    case, T, V = s["case"], s["T"], s["V"]
    op, hard = case["op"], case["hard"]
    z = s["logits"][:, :V].float()
    got = {}
    t = has = None
    if s["targets"] is not None:
        has = s["targets"] >= 0
        t = s["targets"].clamp(min=0)[:, None]
    if op == "logprobs":
        d, total, got["lse"] = _plain_softmax(z, T)
        log_total = total.log()
        e = d.exp()
        # sum p ln p = sum e d / total - ln total; a masked entry has e = 0 and adds nothing
        got["entropy"] = (log_total - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total)[:, 0]
        got["logprob"] = torch.where(has, (d.gather(1, t) - log_total)[:, 0], 0.0)
        if case["top_k"]:
            ids = _plain_top(z, case["top_k"])
            got["top_ids"] = ids.to(torch.int32)
            got["top_logprobs"] = d.gather(1, ids) - log_total
        return got
    if op == "logprobs_grad":
        logp = z / T - s["lse"][:, None]
        p = logp.exp()
        a = torch.where(has, s["d_logprob"], 0.0)[:, None]
        grad = -a * p
        if s["d_entropy"] is not None:
            grad = grad - s["d_entropy"][:, None] * torch.where(
                p > 0, p * (logp + s["entropy"][:, None]), 0.0)
        grad.scatter_add_(1, t, a)
        got["d_logits"] = (grad / T).to(s["logits"].dtype)
        return got
    q, logq, ids = _plain_teacher(s)
    if op == "distill_grad":
        p = (z / T - s["lse"][:, None]).exp()
    else:
        d, total, got["lse"] = _plain_softmax(z, T)
        logp = d.gather(1, ids) - total.log()
        got["loss"] = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
        p = d.exp() / total if op == "distill_loss_grad" else None
    if hard:
        if op == "distill_grad":
            p1 = (z - s["hard_lse"][:, None]).exp()
        else:
            d, total, got["hard_lse"] = _plain_softmax(z, 1.0)
            got["logprob"] = torch.where(has, (d.gather(1, t) - total.log())[:, 0], 0.0)
            p1 = d.exp() / total if op == "distill_loss_grad" else None
    if op != "distill":
        w = s["d_loss"][:, None] / T
        grad = w * q.sum(1, keepdim=True) * p
        grad.scatter_add_(1, ids, -w * q)
        if hard:
            h = torch.where(has, s["d_logprob"], 0.0)[:, None]
            grad -= h * p1
            grad.scatter_add_(1, t, h)
        got["d_logits"] = grad.to(s["logits"].dtype)
    return {name: got[name] for name in _returned(case)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    R, V, K, k = case["rows"], case["vocab"], case["teacher_k"], case["top_k"]
    es = BYTES[case["dtype"]]
    op = case["op"]
    # a gradient pass need not read the rows without weight
    read = R * V * es * ((1.0 - IGNORED) if op in ("logprobs_grad", "distill_grad") else 1.0)
    moved = read + (R * V * es if op.endswith("grad") else 0)
    if s_teacher := K * (4 + BYTES[case["teacher"]]):
        moved += R * (s_teacher + 4 * case["teacher_lse"])
    moved += R * (8 + 16 + 8 * k)
    # subtract, scale, exp, add (and the entropy's multiply-add); a gradient scales, exps, multiplies
    each = {"logprobs": 6, "logprobs_grad": 7, "distill": 4, "distill_grad": 4,
            "distill_loss_grad": 8}[op]
    if case["hard"] and case["temperature"] != 1.0:
        each *= 2
    return {"bytes": float(moved), "flops": float(each) * R * V}


def exact(case, seed):
    s = prepare(case, seed)
    R, V, T, K = s["R"], s["V"], s["T"], case["teacher_k"]
    op, hard = case["op"], case["hard"]
    parts = {}

    def put(name, x):
        parts.setdefault(name, []).append(x)

    def cut(name, i, n):
        return None if s.get(name) is None else s[name][i:i + n]

    n = max(1, min(R, (1 << 27) // V))
    for i in range(0, R, n):
        z = s["logits"][i:i + n, :V].double()
        rows = torch.arange(z.shape[0], device=z.device)
        tgt = cut("targets", i, n)
        some = None if tgt is None else tgt >= 0
        given = op in ("logprobs_grad", "distill_grad")
        lse = cut("lse", i, n).double() if given else torch.logsumexp(z / T, 1)
        logp = (z / T).sub_(lse[:, None])
        if hard:
            lse1 = cut("hard_lse", i, n).double() if given else torch.logsumexp(z, 1)
        if K:
            u = cut("teacher_logits", i, n).double() / T
            ids = cut("teacher_ids", i, n).long()
            u[ids < 0] = -math.inf
            tl = cut("teacher_lse", i, n)
            u -= (torch.logsumexp(u, 1) if tl is None else tl.double())[:, None]
            q = u.exp()
            at = ids.clamp(min=0)
        if not given:
            put("lse", lse)
        if op == "logprobs":
            put("entropy", torch.special.entr(logp.exp()).sum(1))
            put("logprob", torch.where(some, logp[rows, tgt.clamp(min=0)], 0.0))
            if case["top_k"]:
                # in falling order: the values do not depend on how ties are broken
                put("top_logprobs", torch.sort(logp, dim=1, descending=True)
                    .values[:, :case["top_k"]].contiguous())
        elif op in ("distill", "distill_loss_grad"):
            put("loss", torch.where(q > 0, q * (u - logp.gather(1, at)), 0.0).sum(1))
            if hard:
                put("hard_lse", lse1)
                put("logprob", torch.where(some, z[rows, tgt.clamp(min=0)] - lse1, 0.0))
        if op.endswith("grad"):
            p = logp.exp()
            if op == "logprobs_grad":
                a = torch.where(some, cut("d_logprob", i, n).double(), 0.0)
                grad = p * -a[:, None]
                b = cut("d_entropy", i, n)
                if b is not None:
                    inner = logp.add_(cut("entropy", i, n).double()[:, None]).mul_(p)
                    inner[p == 0] = 0.0
                    grad -= b.double()[:, None] * inner
                grad[rows, tgt.clamp(min=0)] += a
                grad /= T
            else:
                w = cut("d_loss", i, n).double() / T
                grad = p.mul_((w * q.sum(1))[:, None])
                grad.scatter_add_(1, at, -w[:, None] * q)
                if hard:
                    h = torch.where(some, cut("d_logprob", i, n).double(), 0.0)
                    grad.sub_(z.sub_(lse1[:, None]).exp_().mul_(h[:, None]))
                    grad[rows, tgt.clamp(min=0)] += h
            # 64 bits where they fit, 32 for the largest gradients (their type has 8 bits)
            put("d_logits", grad if R * V < 1 << 28 else grad.float())
    return {name: torch.cat(parts[name]) if name in parts else None for name in _returned(case)}
