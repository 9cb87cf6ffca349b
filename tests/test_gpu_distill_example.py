"""The distillation example runs, and its step's gradients are the loss's (fp64 differentiation of
the same step)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_the_example_runs():
    first, last, before, after = _example().train(steps=5, log=None)
    for x in (first, last, before, after):
        assert x == x and abs(x) < 100


def test_its_gradients():
    ex = _example()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    d, T, D = ex.Drafter(g), 96, torch.float64
    step = ex.Step(d, T)
    target = 2.5 * torch.randn(ex.V, ex.V, generator=g, device="cuda")
    tokens = torch.randint(ex.V, (T,), generator=g, device="cuda").int()
    total = step(tokens, target[tokens.long()]).item()
    p = [x.to(D).requires_grad_() for x in d.params()]
    table, w1, w2, w_pre = p
    t = tokens.long()
    x = 8.0 * table[t]
    h = x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * (1.0 + w_pre)
    logp = torch.log_softmax(h @ table.t() + w1[t] @ w2, 1)
    z = target[t].to(D)
    lq, ids = torch.log_softmax(z, 1).sort(1, descending=True)
    lq, ids = lq[:, :ex.K], ids[:, :ex.K]
    want = (lq.exp() * (lq - logp.gather(1, ids))).sum(1).mean()
    want.backward()
    # x, h, d_hidden and d_x are rounded to bf16 on the way, each by up to 2^-9 of itself, and the
    # logits' gradient by 2^-9 of each entry: together at most 5 2^-9 of a sum of magnitudes, which
    # for these random signs is some four times the sum itself
    tol = 20 * 2.0 ** -9
    assert abs(total - want.item()) <= 2.0 ** -6 * want.item()
    for got, ref in zip(step.grads, p):
        assert (got.to(D) - ref.grad).norm() <= tol * ref.grad.norm()
