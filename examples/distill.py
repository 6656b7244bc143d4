"""Distil a teacher's recorded top tokens into a small student, sharded over
emulated data-parallel ranks: the losses that make the gradients, and the
shard-local step that consumes them, as a training job calls them.

The student is the two matrices at a language model's ends (an embedding and an
output head, vocabulary 1000, width 256); the teacher a fixed table of logits
for the token that follows. Each step, every rank
  1. records its tokens' 16 most likely successors by the teacher
     (zs_token_logprobs: ids and log probabilities),
  2. takes the loss against that record mixed with the hard labels', and its
     gradient, in one pass over the student's logits, in place
     (zs_distill_loss_grad),
  3. turns it into its flat bf16 gradient (the model's own backward pass; the
     matrix products are torch's),
and then every rank's zs_shard_step takes the mean of the ranks' slices of its
shard, updates it with AdamW and casts it into the flat parameter buffer, whose
views are the student's weights for the next step.

    python examples/distill.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fsdp_sharded_mixed_gb300 as zs  # noqa: E402

VOCAB, WIDTH, WORLD, TOKENS, TOP = 1000, 256, 4, 512, 16
SOFT, HARD = 0.8, 0.2   # weights of the two losses
HPARAMS = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)


def main(steps=60, log=print):
    """Returns the mean distillation loss of the first and the last step, and
    the mean log probability of held-out tokens before and after."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    f32 = dict(dtype=torch.float32, device=dev)

    # What each token is followed by, to the teacher.
    teacher = torch.randn(VOCAB, VOCAB, generator=g, **f32) * 2.5

    plan = zs.zs_flatten_plan([VOCAB * WIDTH, VOCAB * WIDTH], world=WORLD)
    S = plan.S
    params = torch.zeros(plan.P_pad, dtype=torch.bfloat16, device=dev)
    embed, head = (params.narrow(0, off, VOCAB * WIDTH).view(VOCAB, WIDTH)
                   for off in zs.zs_plan_offsets(plan))
    master = torch.zeros(plan.P_pad, **f32)
    master[:plan.P].normal_(0.0, 0.05, generator=g)
    params.copy_(master)
    shards = [[x.narrow(0, r * S, S) for x in
               (master, torch.zeros(plan.P_pad, **f32), torch.zeros(plan.P_pad, **f32))]
              for r in range(WORLD)]
    grads = [torch.zeros(plan.P_pad, dtype=torch.bfloat16, device=dev) for _ in range(WORLD)]

    # A rank's buffers, kept from step to step.
    logits = torch.empty(TOKENS, VOCAB, dtype=torch.bfloat16, device=dev)
    ids = torch.empty(TOKENS, TOP, dtype=torch.int32, device=dev)
    record = torch.empty(TOKENS, TOP, **f32)
    zero_lse = torch.zeros(TOKENS, **f32)   # the record holds log probabilities already
    loss, logprob, entropy = (torch.empty(TOKENS, **f32) for _ in range(3))
    w_soft = torch.full((TOKENS,), SOFT / TOKENS, **f32)
    w_hard = torch.full((TOKENS,), -HARD / TOKENS, **f32)   # of the log probability

    def batch():
        tokens = torch.randint(0, VOCAB, (TOKENS,), generator=g, device=dev)
        following = torch.multinomial(torch.softmax(teacher[tokens], 1), 1, generator=g)[:, 0]
        return tokens, following

    held_out = batch()

    def evaluate():
        tokens, following = held_out
        torch.mm(embed[tokens], head.t(), out=logits)
        zs.zs_token_logprobs(logits, zs.ZS_BF16, TOKENS, VOCAB, VOCAB, following, 1.0, logprob,
                             entropy)
        return logprob.mean().item(), entropy.mean().item()

    before = evaluate()
    log(f"held out: log probability {before[0]:.3f}, entropy {before[1]:.3f}")
    losses = []
    for step in range(1, steps + 1):
        total = 0.0
        for rank in range(WORLD):
            tokens, following = batch()
            zs.zs_token_logprobs(teacher[tokens], zs.ZS_FP32, TOKENS, VOCAB, VOCAB, None, 1.0,
                                 top_k=TOP, top_ids=ids, top_logprobs=record)
            hidden = embed[tokens]
            torch.mm(hidden, head.t(), out=logits)
            zs.zs_distill_loss_grad(logits, zs.ZS_BF16, TOKENS, VOCAB, VOCAB, ids, record,
                                    zs.ZS_FP32, TOP, zero_lse, 1.0, following, w_soft, w_hard,
                                    loss, None, logprob, None, logits, VOCAB)
            total += loss.mean().item()
            d_embed = torch.zeros(VOCAB, WIDTH, **f32)
            d_embed.index_add_(0, tokens, (logits @ head).float())
            flat = grads[rank]
            flat[:VOCAB * WIDTH] = d_embed.flatten()
            flat[VOCAB * WIDTH:plan.P] = (logits.t() @ hidden).flatten()
        for rank, state in enumerate(shards):
            slices = [flat.narrow(0, rank * S, S) for flat in grads]
            zs.zs_shard_step(plan, rank, 0, S, slices, zs.ZS_BF16, *state, params, zs.ZS_BF16,
                             HPARAMS, step)
        losses.append(total / WORLD)
        if step == 1 or step % 10 == 0:
            log(f"step {step}: distillation loss {losses[-1]:.3f}")
    after = evaluate()
    zs.zs_check_device_error()
    log(f"held out: log probability {after[0]:.3f}, entropy {after[1]:.3f}")
    return losses[0], losses[-1], before[0], after[0]


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
