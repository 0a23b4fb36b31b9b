"""A language model small enough to read, trained end to end with the library's calls.

The model is a bigram: the hidden state of a token is its embedding, the head scores
the next one.  N data-parallel ranks each draw their own batch, and every step is

  1. per rank, the loss and the gradients of hidden states and head
     (ss_linear_cross_entropy; the prompt half of each sequence is ignored);
  2. per fully_shard group, the reduce-scatter with its sum of squares
     (fsdp_pack, fsdp_reduce_scatter_norm), as gradients become final;
  3. one norm over all groups, AdamW on the clipped mean (fsdp_clip_adamw);
  4. the all-gather (fsdp_all_gather_unpack).

    python examples/clipped_training.py [--steps 60] [--ranks 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sharded_state_gb300 as ss  # noqa: E402

VOCAB, HIDDEN, BATCH, LENGTH = 500, 96, 8, 64


def batch(gen, follow):
    """Sequences in which token t is mostly followed by follow[t]; the first half of each is a prompt."""
    x = torch.empty(BATCH, LENGTH + 1, dtype=torch.int64, device="cuda")
    x[:, 0] = torch.randint(0, VOCAB, (BATCH,), generator=gen, device="cuda")
    stray = torch.rand(BATCH, LENGTH, generator=gen, device="cuda") < 0.1
    other = torch.randint(0, VOCAB, (BATCH, LENGTH), generator=gen, device="cuda")
    for i in range(LENGTH):
        x[:, i + 1] = torch.where(stray[:, i], other[:, i], follow[x[:, i]])
    targets = x[:, 1:].clone()
    targets[:, :LENGTH // 2] = -100
    return x[:, :-1].reshape(-1), targets.reshape(-1)


def train(steps=60, ranks=4, max_norm=0.1, lr=2e-2, log=print):
    """Returns the mean loss of every step and the number of steps that were clipped."""
    gen = torch.Generator("cuda").manual_seed(0)
    follow = torch.randperm(VOCAB, generator=gen, device="cuda")
    tokens = BATCH * LENGTH
    params = [(torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda") * 0.5).to(torch.bfloat16) for _ in range(2)]
    plan = ss.fsdp_plan_create(ss.SS_PER_PARAM_DIM0, ranks, 2, [VOCAB, VOCAB], [HIDDEN, HIDDEN],
                               group_num_params=[1, 1])
    total = plan.info().total_numel

    shards = torch.empty(total, dtype=torch.bfloat16, device="cuda")
    master, m, v, reduced = (torch.empty(total, device="cuda") for _ in range(4))
    ss.fsdp_pack(plan, params, shards)
    ss.fsdp_init_master(plan, shards, master, m, v)

    packed = [torch.empty(total, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
    grads = [[torch.empty_like(p) for p in params] for _ in range(ranks)]
    d_hidden = torch.empty(tokens, HIDDEN, dtype=torch.bfloat16, device="cuda")
    losses = torch.empty(steps, ranks, device="cuda")
    norms = torch.empty(steps, 2, device="cuda")
    sums = torch.empty(2, dtype=torch.float64, device="cuda")
    loss_ws = torch.empty(ss.ss_linear_ce_workspace(tokens, HIDDEN, VOCAB, True), dtype=torch.uint8, device="cuda")
    norm_ws = torch.empty(ss.SS_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    for step in range(steps):
        embedding, head = params
        for r in range(ranks):
            x, targets = batch(gen, follow)
            ss.ss_linear_cross_entropy(embedding[x], head, targets, losses[step, r:], loss_ws, d_hidden=d_hidden,
                                       d_weight=grads[r][1])
            grads[r][0].copy_(torch.zeros(VOCAB, HIDDEN, device="cuda").index_add_(0, x, d_hidden.float()))
        for group in (1, 0):  # the head's gradient is final first
            for r in range(ranks):
                ss.fsdp_pack(plan, grads[r], packed[r], group=group)
            ss.fsdp_reduce_scatter_norm(plan, packed, reduced, sums[group:], norm_ws, group=group)
        hp = ss.adamw_params(lr=lr, weight_decay=0.0, step=step + 1)
        for group in (0, 1):
            ss.fsdp_clip_adamw(plan, reduced, sums, max_norm, master, m, v, shards, hp, norms[step], group=group)
        ss.fsdp_all_gather_unpack(plan, shards, params)
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {losses[step].mean().item():.3f}  norm {norms[step, 0].item():.3f}  "
                f"factor {norms[step, 1].item():.3f}")
    clipped = int((norms[:, 1] < 1).sum())
    return losses.mean(1).tolist(), clipped


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    train(a.steps, a.ranks)
