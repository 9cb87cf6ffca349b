"""Trains a small drafter with tied embeddings on a target's distribution, and drafts for the
tokens that the target samples.

The target is a table of logits: what follows token t has the probabilities of its row t.  Each
step is what a training program does with the target's logits over a batch:

    top_logits -> embed -> block_norm -> distill_loss -> block_norm_backward
      -> embed_backward (onto the head's gradient: one table is both) -> clip_grads -> SGD (torch)

Afterwards the drafter proposes one token after another, the target's logits are sampled, and
verify counts the drafts that are what was drawn.

    python examples/distill_head.py [--steps 200]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dspark_block_drafter_gb300 import torch_io as tio  # noqa: E402

B, L, H, V, R, K = 64, 4, 128, 512, 64, 32


class Drafter:
    """One table for both ends, and the Markov term of the head."""

    def __init__(self, g):
        def randn(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

        self.table, self.w_pre = randn(V, H, std=0.1), randn(H, std=0.1)
        self.head = tio.Head(self.table, randn(V, R, std=0.1), randn(R, V, std=0.1))

    def params(self):
        return [self.table, self.head.markov_w1, self.head.markov_w2, self.w_pre]


class Step:
    """The buffers of a training step of T rows, and the step."""

    def __init__(self, drafter, T):
        e = dict(dtype=torch.bfloat16, device="cuda")
        self.d = drafter
        self.ecfg = tio.make_embed_config(T, V, H, "bf16", scale=8.0)
        self.ncfg = tio.make_norm_config(T, H, "bf16", weight_offset=1.0)
        self.lcfg = tio.make_loss_config(T, H, V, R, "bf16")
        self.x, self.h = torch.empty(T, H, **e), torch.empty(T, H, **e)
        self.teacher = tio.Teacher(torch.empty(T, K, dtype=torch.int32, device="cuda"),
                                   torch.empty(T, K, device="cuda"), torch.empty(T, device="cuda"))
        self.out = tio.LossOutputs.allocate(self.lcfg, drafter.head)
        self.ngrads = tio.NormGrads.allocate(self.ncfg, gate=False, w_post=False, y=False)
        self.loss_ws = tio.distill_workspace_for(self.lcfg, drafter.head, self.teacher, self.out)
        self.norm_ws = tio.norm_workspace_for(self.ncfg)
        self.embed_ws = tio.embed_workspace_for(self.ecfg)
        # in the order of Drafter.params()
        self.grads = [self.out.d_lm_head, self.out.d_markov_w1, self.out.d_markov_w2,
                      self.ngrads.d_w_pre]

    def hidden(self, tokens):
        tio.embed(self.ecfg, self.d.table, tokens, self.x)
        tio.block_norm(self.ncfg, self.x, None, self.d.w_pre, self.h)
        return self.h

    def __call__(self, tokens, target_logits):
        """The loss's total on the device; self.grads hold the gradients."""
        t = self.teacher
        tio.top_logits(target_logits, t.ids, t.logits, lse=t.lse)
        tio.distill_loss(self.lcfg, self.d.head, t, self.hidden(tokens), tokens, self.out,
                         self.loss_ws)
        tio.block_norm_backward(self.ncfg, self.x, None, self.d.w_pre, self.out.d_hidden, self.ngrads,
                                self.norm_ws)
        tio.embed_backward(self.ecfg, tokens, self.ngrads.d_x, self.out.d_lm_head, self.embed_ws,
                           add=self.out.d_lm_head)
        return self.out.total


def accepted(drafter, step, target, g):
    """Mean accepted length of L drafts a block for the target's sampled tokens."""
    anchors = torch.randint(V, (B,), generator=g, device="cuda").int()
    cfg = tio.make_config(B, 1, H, V, R, 1, True, 0.0, "bf16")
    out = tio.Outputs.allocate(B, 1, 1, V, topk=False, conf=False)
    ws = tio.workspace_for(cfg, drafter.head)
    prev, drafts, sampled = anchors, [], []
    scfg = tio.make_sample_config(B, V, "f32", temperature=0.5, top_p=0.9)
    u = torch.rand(L + 1, B, generator=g, device="cuda")
    follow = anchors
    for i in range(L + 1):
        token = torch.empty(B, dtype=torch.int32, device="cuda")
        tio.sample(scfg, target[follow.long()], u[i], token)
        sampled.append(token)
        follow = token
        if i < L:
            tio.propose(cfg, drafter.head, step.hidden(prev).view(B, 1, H), prev, out, ws)
            prev = out.draft[:, 0].clone()
            drafts.append(prev)
    acc, bonus = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    tio.verify(torch.stack(drafts, 1).contiguous(),
               torch.full((B,), L, dtype=torch.int32, device="cuda"),
               torch.stack(sampled, 1).contiguous(), acc, bonus)
    return acc.float().mean().item()


def train(steps=200, seed=0, log=print):
    """Returns (first loss, last loss, accepted length before, accepted length after)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    target = 2.5 * torch.randn(V, V, generator=g, device="cuda")
    drafter = Drafter(g)
    full = [p.float() for p in drafter.params()]
    T = 512
    step, one = Step(drafter, T), Step(drafter, B)
    clipped = tio.GradList(step.grads)
    clip_ws = tio.clip_workspace_for(clipped)
    norm = torch.empty(1, device="cuda")
    before = accepted(drafter, one, target, g)
    first = None
    for i in range(steps):
        tokens = torch.randint(V, (T,), generator=g, device="cuda").int()
        total = step(tokens, target[tokens.long()])
        tio.clip_grads(clipped, 1.0, norm, clip_ws)
        for p, f, d in zip(drafter.params(), full, step.grads):
            f.sub_(d.float(), alpha=2.0)
            p.copy_(f)
        if first is None:
            first = total.item()
        if log and (i % 50 == 0 or i == steps - 1):
            log(f"step {i:4d}  divergence {total.item():7.4f}  gradient norm {norm.item():.4f}")
    if tio.device_status(step.loss_ws) != 0 or tio.device_status(step.embed_ws) != 0:
        raise RuntimeError("a step failed on the device")
    last = total.item()
    after = accepted(drafter, one, target, g)
    if log:
        log(f"accepted of {L}: {before:.2f} before, {after:.2f} after")
    return first, last, before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    train(ap.parse_args().steps)
