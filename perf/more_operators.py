"""What the operators around a training step's layers are measured on: the
embedding lookup and its gradient, layer norm and its gradient, and the global
norm of a list of gradients with clipping.

Widths, vocabularies and parameter lists are those of the repository's models
(256, 768, 2048, 4096; 1000, 32000, 50257, 151936); rows are tokens of a batch.
``op`` names the call of a case:
  embedding        zs_embedding
  embedding_grad   zs_embedding_grad
  layer_norm       zs_layer_norm
  layer_norm_grad  zs_layer_norm_grad
  clip             zs_tensors_clip
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
EPS = 1e-5
PADDED = 1.0 / 16               # share of tokens that are padding (a negative id)
MOST_TABLE = 152064 * 2048      # elements of a drawn table
MOST_ROWS = 16384 * 4096        # elements of a drawn batch of rows
MOST_LISTED = 3_100_000_000     # elements of a drawn list of gradients, in bf16


def _table(name, op, rows, vocab, dim, dtype, table="bf16", scale=1.0, pad=0, add=False):
    return dict(name=name, op=op, rows=rows, vocab=vocab, dim=dim, dtype=dtype, table=table,
                scale=scale, pad=pad, add=add)


def _norm(name, op, rows, dim, dtype, weight="bf16", residual=False, bias=True, pad=0):
    return dict(name=name, op=op, rows=rows, dim=dim, dtype=dtype, weight=weight,
                residual=residual, bias=bias, pad=pad)


def _clip(name, layers, dim, inner, vocab, narrow, dtype, out="bf16", bias=True, max_norm=1.0):
    return dict(name=name, op="clip", layers=layers, dim=dim, inner=inner, vocab=vocab,
                narrow=narrow, dtype=dtype, out=out, bias=bias, max_norm=max_norm)


def listed():
    return [
        # One sequence's next token: a generation step, all latency.
        _table("embedding one token", "embedding", 1, 50257, 768, "bf16"),
        # A batch of 8 sequences of 2048 tokens, scaled by the root of the width.
        _table("embedding batch", "embedding", 16384, 151936, 2048, "bf16", scale=2048 ** 0.5),
        # The tiny model's step: fp32 gradients of 512 tokens.
        _table("embedding_grad tiny", "embedding_grad", 512, 1000, 256, "bf16", table="fp32"),
        # A tied table's gradient: the head's is there already and the tokens' comes on top.
        _table("embedding_grad tied", "embedding_grad", 8191, 50257, 768, "bf16", add=True),
        # A batch against the largest vocabulary.
        _table("embedding_grad batch", "embedding_grad", 16384, 151936, 2048, "bf16",
               scale=2048 ** 0.5),
        # The same generation step's norm behind its residual sum.
        _norm("layer_norm one token", "layer_norm", 1, 768, "bf16", residual=True),
        # A batch's norm behind its residual sum, fp32 weights.
        _norm("layer_norm batch", "layer_norm", 16384, 4096, "bf16", weight="fp32",
              residual=True),
        # A small batch's backward pass: the sums over the rows count.
        _norm("layer_norm_grad small", "layer_norm_grad", 1023, 768, "fp32", weight="fp32"),
        # A batch's backward pass with the gradient that goes past the norm.
        _norm("layer_norm_grad batch", "layer_norm_grad", 16384, 4096, "bf16", residual=True),
        # The tiny model's list of gradients.
        _clip("clip tiny", 2, 256, 1024, 1000, 256, "fp32", out="fp32"),
        # A list of 148 gradients, clipped into the flat buffer: fp32 sums, bf16 slices.
        _clip("clip list", 12, 768, 4 * 768, 50257, 768, "fp32"),
        # The largest list: 3.09 billion elements.
        _clip("clip large list", 36, 2048, 11008, 151936, 256, "bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, an odd one at times."""
    d = _log_uniform(rng, lo, hi)
    return d if rng.random() < 0.35 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "layer_norm", "layer_norm_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    pad = rng.choice([0, 0, 0, 1, 64])
    other = rng.choice(["bf16", "fp32"])
    if op.startswith("embedding"):
        dim = _width(rng, 64, 8192)
        fit = 1 if "fp32" not in (dtype, other) else 2
        vocab = _log_uniform(rng, 256, min(151936, MOST_TABLE // dim // fit))
        rows = _log_uniform(rng, 1, min(32768, MOST_ROWS // dim // fit))
        case = _table("", op, rows, vocab, dim, dtype, other,
                      rng.choice([1.0, dim ** 0.5, round(rng.uniform(0.1, 8.0), 3)]), pad,
                      op == "embedding_grad" and rng.random() < 0.4)
    elif op.startswith("layer_norm"):
        dim = _width(rng, 64, 16384)
        rows = _log_uniform(rng, 1, min(32768, MOST_ROWS // dim // (BYTES[dtype] // 2)))
        case = _norm("", op, rows, dim, dtype, other, rng.random() < 0.6, rng.random() < 0.8, pad)
    else:
        layers, dim = _log_uniform(rng, 1, 40), _width(rng, 64, 2048)
        inner = dim * rng.choice([2, 4]) + rng.choice([0, 0, 17])
        vocab, narrow = _log_uniform(rng, 256, 151936), _log_uniform(rng, 16, dim)
        one = 2 * dim * dim + 2 * dim * narrow + 3 * dim * inner
        most = MOST_LISTED // (BYTES[dtype] // 2) - vocab * dim
        layers = max(1, min(layers, most // one))
        case = _clip("", layers, dim, inner, vocab, narrow, dtype, other, rng.random() < 0.5,
                     rng.choice([1.0, 0.5, round(rng.uniform(0.05, 2.0), 3)]))
    del case["name"]
    return case


def _numels(case):
    """The lengths of a model's gradients in the order of its modules: the
    table, then by layer two norms, the attention's four matrices, the three of
    the gated layer (biases with them), and the last norm."""
    d, f, n = case["dim"], case["inner"], case["narrow"]
    layer = []
    for rows, cols in ((d, 0), (d, d), (n, d), (n, d), (d, d), (d, 0), (f, d), (f, d), (d, f)):
        layer.append(rows * cols if cols else rows)
        if case["bias"]:
            layer.append(rows)
    return [case["vocab"] * d] + layer * case["layers"] + [d]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + case["dim"] * 7 + case.get("rows", 0))
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, sigma, generator=g)

    s = dict(case=case)
    if op == "clip":
        numels = _numels(case)
        total = sum(numels)
        # backward leaves each gradient in a tensor of its own; a few entries are large
        grads = [normal(n, sigma=1e-3, dtype=dt) for n in numels]
        for x in grads[:: 7]:
            x[:: 97] *= 30.0
        s["grads"] = grads
        # the flat gradient buffer and each tensor's place in it
        s["flat"] = torch.empty(total, dtype=DTYPES[case["out"]], device=dev)
        s["outs"] = list(torch.split(s["flat"], numels))
        s["workspace"] = torch.empty(1 << 16, dtype=torch.uint8, device=dev)
        s["norm"], s["coef"] = (torch.empty(1, device=dev) for _ in range(2))
        s["nonfinite"] = torch.empty(1, dtype=torch.int32, device=dev)
        if own:  # the addresses of buffers that live as long as the program, marshalled once
            import fsdp_sharded_mixed_gb300 as zs
            s["in_list"], s["out_list"] = zs.Tensors(grads), zs.Tensors(s["outs"])
        return s
    R, D = case["rows"], case["dim"]
    ld = D + case["pad"]
    if op.startswith("embedding"):
        V, tt = case["vocab"], DTYPES[case["table"]]
        # few tokens are frequent, most are rare: the k-th as often as 1/k
        u = torch.rand(R, generator=g, device=dev, dtype=torch.float64)
        tokens = ((V + 1.0) ** u).long().sub_(1).clamp_(0, V - 1)
        s["tokens"] = torch.where(torch.rand(R, generator=g, device=dev) < PADDED, -1, tokens)
        if op == "embedding":
            s["table"] = normal(V, D, sigma=0.02, dtype=tt)
            s["out"] = torch.empty(R, ld, dtype=dt, device=dev)
        else:
            s["d_out"] = normal(R, ld, sigma=1e-3, dtype=dt)
            s["add"] = normal(V, D, sigma=1e-3, dtype=tt) if case["add"] else None
            s["d_table"] = torch.empty(V, D, dtype=tt, device=dev)
            # sorted tokens, long runs' parts
            s["workspace"] = torch.empty((1 << 21) + 24 * R + 4 * (R // 16 + 2) * D,
                                         dtype=torch.uint8, device=dev)
        return s
    wt = DTYPES[case["weight"]]
    s["weight"] = (1.0 + normal(D, sigma=0.1)).to(wt)
    s["bias"] = normal(D, sigma=0.1, dtype=wt) if case["bias"] else None
    # a residual stream: a few features far larger than the others, an offset
    feature = torch.where(torch.rand(D, generator=g, device=dev) < 0.01, 8.0, 1.0)

    def stream(sigma):
        x = torch.empty(R, ld, dtype=dt, device=dev)
        for i in range(0, R, 2048):
            r = min(2048, R - i)
            x[i:i + r] = 0.0
            x[i:i + r, :D] = normal(r, D) * (sigma * feature) + 0.2 * sigma
        return x

    s["x"] = stream(1.5)
    if op == "layer_norm":
        s["residual"] = stream(1.0) if case["residual"] else None
        s["sum"] = torch.empty(R, ld, dtype=dt, device=dev) if case["residual"] else None
        s["y"] = torch.empty(R, ld, dtype=dt, device=dev)
        s["mean"], s["rstd"] = (torch.empty(R, device=dev) for _ in range(2))
        return s
    # what the forward pass left
    s["mean"], s["rstd"] = (torch.empty(R, device=dev) for _ in range(2))
    for i in range(0, R, 1024):
        x = s["x"][i:i + 1024, :D].double()
        s["mean"][i:i + 1024] = x.mean(1)
        s["rstd"][i:i + 1024] = (x.var(1, unbiased=False) + EPS).rsqrt()
    s["d_y"] = normal(R, ld, sigma=1e-3, dtype=dt)
    s["d_sum"] = normal(R, ld, sigma=1e-3, dtype=dt) if case["residual"] else None
    s["d_x"] = torch.empty(R, ld, dtype=dt, device=dev)
    s["d_weight"] = torch.empty(D, dtype=wt, device=dev)
    s["d_bias"] = torch.empty(D, dtype=wt, device=dev) if case["bias"] else None
    # one part of both sums for each group of rows
    s["workspace"] = torch.empty((1 << 16) + 2 * 4 * 1216 * D, dtype=torch.uint8, device=dev)
    return s


def _run_own(s):
    import fsdp_sharded_mixed_gb300 as zs
    code = {"bf16": zs.ZS_BF16, "fp32": zs.ZS_FP32}
    case = s["case"]
    op, dtype, D = case["op"], code[case["dtype"]], case["dim"]
    if op == "clip":
        zs.zs_tensors_clip(s["in_list"], dtype, case["max_norm"], s["out_list"],
                           code[case["out"]], s["workspace"], s["norm"], s["coef"],
                           s["nonfinite"])
        return dict(flat=s["flat"], norm=s["norm"], coef=s["coef"], nonfinite=s["nonfinite"])
    R, ld = case["rows"], D + case["pad"]
    if op == "embedding":
        zs.zs_embedding(s["table"], code[case["table"]], case["vocab"], D, D, s["tokens"], R,
                        case["scale"], s["out"], dtype, ld)
        return s["out"][:, :D]
    if op == "embedding_grad":
        zs.zs_embedding_grad(s["d_out"], dtype, R, D, ld, s["tokens"], case["vocab"],
                             case["scale"], s["add"], s["workspace"], s["d_table"],
                             code[case["table"]], D)
        return s["d_table"]
    wt = code[case["weight"]]
    if op == "layer_norm":
        zs.zs_layer_norm(s["x"], dtype, R, D, ld, s["residual"], s["weight"], s["bias"], wt, EPS,
                         s["sum"], s["y"], ld, s["mean"], s["rstd"])
        got = dict(y=s["y"][:, :D], mean=s["mean"], rstd=s["rstd"])
        return dict(got, sum=s["sum"][:, :D]) if case["residual"] else got
    zs.zs_layer_norm_grad(s["d_y"], s["x"], dtype, R, D, ld, ld, s["weight"], wt, s["mean"],
                          s["rstd"], s["d_sum"], s["workspace"], s["d_x"], s["d_weight"],
                          s["d_bias"], wt)
    got = dict(d_x=s["d_x"][:, :D], d_weight=s["d_weight"])
    return dict(got, d_bias=s["d_bias"]) if case["bias"] else got


def _run_plain(s):
    case = s["case"]
    op, dt, D = case["op"], DTYPES[case["dtype"]], case["dim"]
    if op == "clip":
        # a long sum: 64 bits
        total = torch.stack([x.float().square().sum(dtype=torch.float64)
                             for x in s["grads"]]).sum()
        norm = total.sqrt()
        bad = ~torch.isfinite(norm)
        coef = torch.where(bad, 1.0, (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)).float()
        flat = torch.cat([(x.float() * coef).to(DTYPES[case["out"]]) for x in s["grads"]])
        return dict(flat=flat, norm=norm.float().reshape(1), coef=coef.reshape(1),
                    nonfinite=bad.to(torch.int32).reshape(1))
    if op == "embedding":
        tokens = s["tokens"]
        rows = s["table"][tokens.clamp(min=0)].float() * case["scale"]
        return torch.where(tokens[:, None] >= 0, rows, 0.0).to(dt)
    if op == "embedding_grad":
        tokens, tt = s["tokens"], DTYPES[case["table"]]
        total = torch.zeros(case["vocab"], D, device=tokens.device)
        d = torch.where(tokens[:, None] >= 0, s["d_out"][:, :D].float(), 0.0)
        total.index_add_(0, tokens.clamp(min=0), d)
        total = total * case["scale"]
        return (total if s["add"] is None else s["add"].float() + total).to(tt)
    x = s["x"][:, :D].float()
    w = s["weight"].float()
    if op == "layer_norm":
        got = {}
        if case["residual"]:
            # the sum is the stored one: the backward pass sees no other
            got["sum"] = (x + s["residual"][:, :D].float()).to(dt)
            x = got["sum"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / (d.square().mean(1, keepdim=True) + EPS).sqrt()
        y = d * rstd * w
        if case["bias"]:
            y = y + s["bias"].float()
        return dict(got, y=y.to(dt), mean=mean[:, 0], rstd=rstd[:, 0])
    dy = s["d_y"][:, :D].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + s["d_sum"][:, :D].float()
    wt = DTYPES[case["weight"]]
    got = dict(d_x=dx.to(dt), d_weight=(dy * xh).sum(0).to(wt))
    return dict(got, d_bias=dy.sum(0).to(wt)) if case["bias"] else got


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, es, D = case["op"], BYTES[case["dtype"]], case["dim"]
    if op == "clip":
        n = sum(_numels(case))
        return {"bytes": float(n) * (es + BYTES[case["out"]]), "flops": 3.0 * n}
    R = case["rows"]
    if op.startswith("embedding"):
        V, ts = case["vocab"], BYTES[case["table"]]
        live = R * (1.0 - PADDED)
        if op == "embedding":
            # the tokens drawn as 1/k meet this many rows of the table
            met = sum(1.0 - math.exp(-live * p) * 1.0 for p in _shares(V))
            return {"bytes": R * 8.0 + min(met, live) * D * ts + float(R) * D * es,
                    "flops": live * D}
        moved = R * 8.0 + live * D * es + float(V) * D * ts * (2 if case["add"] else 1)
        return {"bytes": moved, "flops": live * D}
    ws = BYTES[case["weight"]]
    if op == "layer_norm":
        rows = 2 + 2 * case["residual"]
        return {"bytes": float(R) * (rows * D * es + 8) + D * ws * (1 + case["bias"]),
                "flops": float(R) * D * (7 + case["residual"] + case["bias"])}
    rows = 3 + case["residual"]
    return {"bytes": float(R) * (rows * D * es + 8) + D * ws * (2 + case["bias"]),
            "flops": float(R) * D * (13 + case["residual"] + case["bias"])}


def _shares(V):
    """The tokens' probabilities, as prepare() draws them."""
    whole = math.log(V + 1.0)
    return [math.log((k + 2.0) / (k + 1.0)) / whole for k in range(V)]


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "clip":
        n = sum(x.numel() for x in s["grads"])
        squares = 0.0
        for x in s["grads"]:
            for part in x.split(1 << 28):
                part = part.double()
                squares += torch.dot(part, part).item()
        norm = math.sqrt(squares)
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        # 64 bits where they fit
        wide = torch.float64 if n < 1 << 29 else torch.float32
        flat = torch.empty(n, dtype=wide, device="cuda")
        at = 0
        for x in s["grads"]:
            flat[at:at + x.numel()] = x.double().mul_(coef)
            at += x.numel()
        one = dict(dtype=torch.float64, device="cuda")
        return dict(flat=flat, norm=torch.tensor([norm], **one), coef=torch.tensor([coef], **one),
                    nonfinite=torch.zeros(1, dtype=torch.int32, device="cuda"))
    R = case["rows"]
    if op == "embedding":
        out = torch.zeros(R, D, dtype=torch.float64, device="cuda")
        some = (s["tokens"] >= 0).nonzero()[:, 0]
        out[some] = s["table"].index_select(0, s["tokens"][some]).double().mul_(case["scale"])
        return out
    if op == "embedding_grad":
        # sums over sorted tokens: differences of running sums would lose digits, so by row
        some = (s["tokens"] >= 0).nonzero()[:, 0]
        out = torch.zeros(case["vocab"], D, dtype=torch.float64, device="cuda")
        out.index_put_((s["tokens"][some],), s["d_out"][some, :D].double().mul_(case["scale"]),
                       accumulate=True)
        return out if s["add"] is None else out.add_(s["add"])
    w = s["weight"].double()
    parts, sums = {}, [torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2)]
    for i in range(0, R, 1024):
        x = s["x"][i:i + 1024, :D].double()
        if op == "layer_norm":
            if case["residual"]:
                x = x.add_(s["residual"][i:i + 1024, :D])
                parts.setdefault("sum", []).append(x)
                x = x.to(s["x"].dtype).double()
            var, mean = torch.var_mean(x, 1, unbiased=False)
            rstd = (var + EPS).rsqrt()
            y = torch.addcmul(s["bias"].double() if case["bias"] else torch.zeros_like(w),
                              (x - mean[:, None]) * rstd[:, None], w)
            for name, v in (("y", y), ("mean", mean), ("rstd", rstd)):
                parts.setdefault(name, []).append(v)
            continue
        dy, r = s["d_y"][i:i + 1024, :D].double(), s["rstd"][i:i + 1024].double()[:, None]
        xh = x.sub_(s["mean"][i:i + 1024].double()[:, None]).mul_(r)
        sums[0] += torch.einsum("rd,rd->d", dy, xh)
        sums[1] += dy.sum(0)
        g = dy.mul_(w)
        along = torch.einsum("rd,rd->r", g, xh)[:, None] / D
        dx = (g - g.sum(1, keepdim=True) / D - xh * along).mul_(r)
        if case["residual"]:
            dx.add_(s["d_sum"][i:i + 1024, :D])
        parts.setdefault("d_x", []).append(dx)
    got = {name: torch.cat(p) for name, p in parts.items()}
    if op == "layer_norm_grad":
        got["d_weight"] = sums[0]
        if case["bias"]:
            got["d_bias"] = sums[1]
    return got
