"""Trains a small drafter head and drafts with it.

The task: token t is always followed by next[t].  The hidden states know nothing of the
tokens, so only the Markov term can learn it.  Each step is what a training program does:

    block_norm -> head_loss -> block_norm_backward -> clip_grads -> Adam (torch)

with teacher-forced previous tokens; afterwards the trained head drafts blocks greedily
from their anchors alone, and verify counts the tokens that hold.

    python examples/train_head.py [--steps 300]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dspark_block_drafter_gb300 import torch_io as tio  # noqa: E402

B, L, H, V, R = 64, 8, 256, 512, 64


class Adam:
    """fp32 copies of bf16 parameters, updated from clipped bf16 gradients."""

    def __init__(self, params, lr):
        self.params, self.lr, self.t = params, lr, 0
        self.full = [p.float() for p in params]
        self.m = [torch.zeros_like(f) for f in self.full]
        self.v = [torch.zeros_like(f) for f in self.full]

    def step(self, grads):
        self.t += 1
        for p, f, m, v, g in zip(self.params, self.full, self.m, self.v, grads):
            g = g.float()
            m.mul_(0.9).add_(g, alpha=0.1)
            v.mul_(0.99).addcmul_(g, g, value=0.01)
            f.sub_(self.lr * (m / (1 - 0.9 ** self.t))
                   / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8))
            p.copy_(f)


def draft(head, hidden, anchors, target):
    """Mean accepted length of greedy drafts from `anchors`."""
    cfg = tio.make_config(B, L, H, V, R, 1, True, 0.0, "bf16")
    head = tio.Head(head.lm_head, head.markov_w1, head.markov_w2).prepare(cfg)
    out = tio.Outputs.allocate(B, L, 1, V, topk=False, conf=False)
    ws = tio.workspace_for(cfg, head)
    tio.propose(cfg, head, hidden, anchors, out, ws)
    accepted = torch.empty(B, dtype=torch.int32, device="cuda")
    bonus = torch.empty_like(accepted)
    tio.verify(out.draft, out.n_draft, target, accepted, bonus)
    if tio.device_status(ws) != 0:
        raise RuntimeError("the draft failed on the device")
    return accepted.float().mean().item()


def train(steps=300, seed=0, log=print):
    """Returns (first loss, last loss, accepted length before, accepted length after)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    follows = torch.randperm(V, generator=g, device="cuda")
    head = tio.Head(randn(V, H, std=0.02), randn(V, R, std=0.1), randn(R, V, std=0.1))
    w_pre, w_post = randn(H, std=0.1), randn(H, std=0.1)     # about 0: weight_offset is 1

    T = B * L
    norm_cfg = tio.make_norm_config(T, H, "bf16", residual_scale=0.5, weight_offset=1.0)
    loss_cfg = tio.make_loss_config(T, H, V, R, "bf16", reduction="mean")
    out = tio.LossOutputs.allocate(loss_cfg, head)
    loss_ws = tio.loss_workspace_for(loss_cfg, head, out)
    ngrads = tio.NormGrads.allocate(norm_cfg, gate=False)
    norm_ws = tio.norm_workspace_for(norm_cfg)
    hidden = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    params = [head.lm_head, head.markov_w1, head.markov_w2, w_pre, w_post]
    raw = [out.d_lm_head, out.d_markov_w1, out.d_markov_w2, ngrads.d_w_pre, ngrads.d_w_post]
    clipped = tio.GradList(raw)                              # in place
    clip_ws = tio.clip_workspace_for(clipped)
    norm = torch.empty(1, device="cuda")
    adam = Adam(params, lr=0.01)

    def blocks():
        """Anchors, their continuations, and a block's inputs."""
        anchors = torch.randint(V, (B,), generator=g, device="cuda")
        tokens = [anchors]
        for _ in range(L + 1):
            tokens.append(follows[tokens[-1]])
        tokens = torch.stack(tokens, 1).int()                # [B, L + 2]
        return tokens, randn(T, H), randn(T, H)

    def inputs(x, y):
        tio.block_norm(norm_cfg, x, y, w_pre, hidden, w_post=w_post)
        return hidden

    tokens, x, y = blocks()
    test = (tokens[:, 0].contiguous(), tokens[:, 1:].contiguous(), x, y)
    before = draft(head, inputs(test[2], test[3]).view(B, L, H), test[0], test[1])
    first = None
    for step in range(steps):
        tokens, x, y = blocks()
        prev = tokens[:, :L].reshape(-1).contiguous()
        labels = tokens[:, 1:L + 1].reshape(-1).contiguous()
        inputs(x, y)
        tio.head_loss(loss_cfg, head, hidden, prev, labels, out, loss_ws)
        tio.block_norm_backward(norm_cfg, x, y, w_pre, out.d_hidden, ngrads, norm_ws,
                                w_post=w_post)
        tio.clip_grads(clipped, 1.0, norm, clip_ws)
        adam.step(raw)
        if first is None:
            first = out.total.item()
        if log and (step % 50 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {out.total.item():7.4f}  gradient norm {norm.item():.4f}")
    if tio.device_status(loss_ws) != 0:
        raise RuntimeError("the loss failed on the device")
    last = out.total.item()
    after = draft(head, inputs(test[2], test[3]).view(B, L, H), test[0], test[1])
    if log:
        log(f"accepted of {L}: {before:.2f} before, {after:.2f} after")
    return first, last, before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=300)
    train(ap.parse_args().steps)
