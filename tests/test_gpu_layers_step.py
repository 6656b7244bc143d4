"""The operators around the layers run together, as a training step runs them:
token and position rows looked up, their sum normalised, cross entropy over a tied
head, the norm's backward pass, the table's gradient added to the head's, all
gradients clipped into the flat buffer, and the shard-local step that consumes it.
The gradients are compared with 64-bit automatic differentiation of the same
model, the steps with the oracle."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import layers_reference as ref
import oracle
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F = zs.ZS_FP32
V, D, SEQ, BATCH, WORLD = 101, 64, 35, 4, 2
R, SCALE, LN_EPS, MAX_NORM = SEQ * BATCH, 2.0, 1e-5, 0.25
NAMES = ("table", "positions", "weight", "bias")
SHAPES = ((V, D), (SEQ, D), (D,), (D,))
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def _batch(seed):
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, V, (R,), generator=g)
    targets = torch.randint(0, V, (R,), generator=g)
    tokens[::11] = -1      # padding, which is not a target either
    targets[::11] = -1
    return tokens, targets


def _reference(params, tokens, targets):
    """Gradients by automatic differentiation in 64 bits, and the largest sum of
    absolute products behind a logit."""
    p = {k: v.double().requires_grad_() for k, v in params.items()}
    rows = torch.where((tokens >= 0)[:, None], SCALE * p["table"][tokens.clamp(min=0)], 0.0)
    h = rows + p["positions"][torch.arange(R) % SEQ]
    y = torch.nn.functional.layer_norm(h, (D,), p["weight"], p["bias"], LN_EPS)
    logp = torch.log_softmax(y @ p["table"].t(), 1)
    live = targets >= 0
    loss = -logp[live, targets[live]].sum() / R
    grads = torch.autograd.grad(loss, list(p.values()))
    return dict(zip(p, grads)), (y.abs() @ p["table"].abs().t()).max().item()


def _step(params, tokens, targets, s):
    """The gradients of a rank, in tensors of their own."""
    pos = torch.arange(R, device=DEV) % SEQ
    zs.zs_embedding(params["table"], F, V, D, D, tokens, R, SCALE, s["e"], F, D)
    zs.zs_embedding(params["positions"], F, SEQ, D, D, pos, R, 1.0, s["p"], F, D)
    # the sum takes the place of the position rows
    zs.zs_layer_norm(s["e"], F, R, D, D, s["p"], params["weight"], params["bias"], F, LN_EPS,
                     s["p"], s["y"], D, s["mean"], s["rstd"])
    logits = s["y"] @ params["table"].t()
    zs.zs_distill_loss_grad(logits, F, R, V, V, None, None, F, 0, None, 1.0, targets, None,
                            s["w"], None, None, s["logprob"], None, logits, V)
    g = {k: torch.empty_like(v) for k, v in params.items()}
    dy = logits @ params["table"]
    g["table"] = logits.t() @ s["y"]
    zs.zs_layer_norm_grad(dy, s["p"], F, R, D, D, D, params["weight"], F, s["mean"], s["rstd"],
                          None, s["ws"], dy, g["weight"], g["bias"], F)
    zs.zs_embedding_grad(dy, F, R, D, D, tokens, V, SCALE, g["table"], s["ws"], g["table"], F, D)
    zs.zs_embedding_grad(dy, F, R, D, D, pos, SEQ, 1.0, None, s["ws"], g["positions"], F, D)
    return g


def test_a_training_step(orc):
    numels = [math.prod(x) for x in SHAPES]
    plan = zs.zs_flatten_plan(numels, world=WORLD)
    offsets, S = zs.zs_plan_offsets(plan), plan.S
    g = torch.Generator(device=DEV).manual_seed(0)
    flat = torch.zeros(plan.P_pad, device=DEV)
    params = {k: flat.narrow(0, o, n).view(x)
              for k, o, n, x in zip(NAMES, offsets, numels, SHAPES)}
    for k, sigma in zip(NAMES, (0.3, 0.3, 0.1, 0.1)):
        params[k].normal_(0.0, sigma, generator=g)
    params["weight"] += 1.0
    master = flat.clone()
    state = [master, torch.zeros_like(flat), torch.zeros_like(flat)]
    o_state = [x.cpu().numpy().copy() for x in state]
    s = {k: torch.empty(R, D, device=DEV) for k in ("e", "p", "y")}
    s["mean"], s["rstd"], s["logprob"] = torch.empty(3, R, device=DEV)
    s["w"] = torch.full((R,), -1.0 / R, device=DEV)
    s["ws"] = torch.empty(max(zs.zs_embedding_grad_workspace_bytes(R, D),
                              zs.zs_layer_norm_grad_workspace_bytes(R, D),
                              zs.zs_grad_norm_workspace_bytes()), dtype=torch.uint8, device=DEV)
    grads = [torch.zeros(plan.P_pad, device=DEV) for _ in range(WORLD)]
    norm, coef = torch.empty(2, 1, device=DEV)
    bad = torch.empty(1, dtype=torch.int32, device=DEV)
    for step in (1, 2, 3):
        host = {k: v.cpu() for k, v in params.items()}
        for rank in range(WORLD):
            tokens, targets = _batch(10 * step + rank)
            got = _step(params, tokens.to(DEV), targets.to(DEV), s)
            want, amp = _reference(host, tokens, targets)
            # a logit is a chain of D products, its error moves a probability by as much and
            # reaches every gradient; then chains over V columns and R rows; the sums'
            # cancellation takes a factor of four at most of these random gradients
            tol = 4 * ref.EPS * (2 * (D + 8) * amp + V + R + 200)
            for k in NAMES:
                off = (got[k].double().cpu() - want[k]).norm() / want[k].norm()
                assert off <= tol, (step, rank, k, off, tol)
            outs = [grads[rank].narrow(0, o, n).view(x)
                    for o, n, x in zip(offsets, numels, SHAPES)]
            zs.zs_tensors_clip([got[k] for k in NAMES], F, MAX_NORM, outs, F, s["ws"], norm, coef,
                               bad)
            exact = math.sqrt(ref.sqnorm([got[k].cpu() for k in NAMES]))
            assert abs(norm.item() - exact) <= (ref.T_SQNORM / 2 + ref.EPS) * exact
            assert exact > MAX_NORM and bad.item() == 0
            for k, out in zip(NAMES, outs):
                assert torch.equal(out, got[k] * coef), k
        for rank in range(WORLD):
            lo, hi = rank * S, (rank + 1) * S
            zs.zs_shard_step(plan, rank, 0, S, [x[lo:hi] for x in grads], F,
                             *[x[lo:hi] for x in state], flat, F, HP, step)
            o_full = np.zeros(plan.P_pad, np.float32)
            part = [x[lo:hi].copy() for x in o_state]
            orc.shard_step(world=WORLD, rank=rank, S=S, lo=0, hi=S,
                           grads=[x[lo:hi].cpu().numpy() for x in grads], master=part[0],
                           m=part[1], v=part[2], full_flat=o_full, lr=HP["lr"], beta1=HP["beta1"],
                           beta2=HP["beta2"], eps=HP["eps"], wd=HP["weight_decay"], t=step,
                           param_dtype=oracle.FP32)
            for mine, theirs in zip(o_state, part):
                mine[lo:hi] = theirs
        assert np.array_equal(state[0].cpu().numpy(), o_state[0])
        assert torch.equal(flat[:plan.P], state[0][:plan.P])   # the next step's weights
    zs.zs_check_device_error()
    plan.free()
