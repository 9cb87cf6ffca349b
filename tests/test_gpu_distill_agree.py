"""Distillation from lists in any order, and gradients of heads that agree with their teacher, to the
digits of the gradient itself.

Bounds, with g = p - q the logits' gradient (the q of a row sum to 1; 0 where a token is not listed):
  - a logit is off by dz (2^-21 of the largest sum of its terms' magnitudes, and 2^-20), which moves
    a log p by twice that and a probability by as much of itself;
  - a listed entry q (e^-x - 1) is off by q times what x = log q - log p is off by: 2 dz, and six
    roundings of numbers no larger than |a| + |log q| + |log p|, 2^-21 of them;
  - the most probable listed token's x is made of two small numbers, -log p as the log1p of the
    other logits' weights and -log q as the log1p of the other listed ones': off by as much of
    *themselves*;
  - bf16 heads round the entries to bf16, from numerators of 11 bits: 2^-8 + 2^-11 of |g|;
  - the products are off by 2^-19 of the sum of their terms' magnitudes, and their results are
    rounded once.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _np(t):
    return t.double().cpu().numpy()


def _tensor(rng, *shape, std=1.0, dtype="f32"):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).cuda().to(DT[dtype])


def _run(h, W, ids, s, dtype, pieces):
    from dspark_block_drafter_gb300 import torch_io as tio
    head = tio.Head(W, None, None, None, None)
    cfg = tio.make_loss_config(h.shape[0], h.shape[1], W.shape[0], 0, dtype, "sum",
                               vocab_pieces=pieces)
    out = tio.LossOutputs.allocate(cfg, head)
    teacher = tio.Teacher(torch.from_numpy(ids).cuda(), torch.from_numpy(s).cuda())
    ws = tio.distill_workspace_for(cfg, head, teacher, out)
    ws.fill_(0xFF)
    tio.distill_loss(cfg, head, teacher, h, None, out, ws)
    torch.cuda.synchronize()
    assert tio.device_status(ws) == 0
    return out


def _check(out, h, W, ids, s, dtype, small):
    """`small`: the most probable token's entry is held to its own digits."""
    x, w = _np(h), _np(W)
    z = x @ w.T
    T, V = z.shape
    rows = np.arange(T)[:, None]
    dz = (np.abs(x) @ np.abs(w).T).max() * 2.0 ** -21 + 2.0 ** -20
    top = z.argmax(1)[:, None]
    d = np.exp(z - z[rows, top])
    others = np.where(np.arange(V) == top, 0.0, d).sum(1, keepdims=True)
    logp = z - z[rows, top] - np.log1p(others)
    a = s.astype(np.float64)
    ta = a.argmax(1)[:, None]
    e = np.exp(a - a[rows, ta])
    rest = np.where(np.arange(a.shape[1]) == ta, 0.0, e).sum(1, keepdims=True)
    lq = a - a[rows, ta] - np.log1p(rest)
    q, p, lp = np.exp(lq), np.exp(logp), logp[rows, ids]
    off = q * (2 * dz + 2.0 ** -21 * (np.abs(a) + np.abs(lq) + np.abs(lp)))
    if small:
        assert np.all(ids[rows, ta] == top)
        at = (rows, ta)
        off[at] = (q * (np.abs(lq) + np.abs(lp)) * (2 * dz + 2.0 ** -19))[at]
    want = (q * (lq - lp)).sum(1)
    each = off.sum(1) + 2.0 ** -21 * (q * np.abs(lq - lp)).sum(1)
    got = _np(out.loss)
    assert np.all(np.abs(got - want) <= each), np.max(np.abs(got - want) / each)
    # expm1 keeps the digits of what is left of two nearly equal probabilities
    g = p.copy()
    g[rows, ids] = q * np.expm1(lp - lq)
    bound = p * (2 * dz + 2.0 ** -18)
    bound[rows, ids] = off * np.maximum(1.0, p[rows, ids] / q)
    bound += np.abs(g) * (2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 0.0)
    for name, m, terms, of in (("d_hidden", g @ w, np.abs(g) @ np.abs(w), bound @ np.abs(w)),
                               ("d_lm_head", g.T @ x, np.abs(g).T @ np.abs(x), bound.T @ np.abs(x))):
        t = getattr(out, name)
        far = np.abs(_np(t) - m)
        most = (of + 2.0 ** -19 * terms) * (1 + OUT[dtype]) + OUT[dtype] * np.abs(m) + 1e-38
        assert np.all(far <= most), (name, np.max(far / most))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,pieces", [(24, 0), (24, 3), (100, 0), (100, 3)])
@pytest.mark.parametrize("order", ["falling", "rising", "shuffled"])
def test_head_that_agrees_with_its_teacher_entry_by_entry(order, T, pieces, dtype):
    """What is left of two equal probabilities is small beside them, and so is its error."""
    rng = np.random.default_rng(T)
    H, V = 64, 512
    W, h = _tensor(rng, V, H, std=0.3, dtype=dtype), _tensor(rng, T, H, dtype=dtype)
    z = _np(h) @ _np(W).T
    k = 256
    ids = np.argsort(-z, axis=1)[:, :k]
    if order == "rising":
        ids = ids[:, ::-1]
    if order == "shuffled":
        ids = rng.permuted(ids, axis=1)
    ids = ids.astype(np.int32).copy()
    s = np.take_along_axis(z, ids, 1).astype(np.float32)
    _check(_run(h, W, ids, s, dtype, pieces), h, W, ids, s, dtype, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,pieces", [(24, 0), (24, 3), (100, 0), (100, 3)])
@pytest.mark.parametrize("order", ["falling", "rising", "shuffled"])
def test_head_that_agrees_with_a_sure_teacher(order, T, pieces, dtype):
    """Head and teacher give one token nearly all: the gradient is of the size of what is left,
    wherever in the list the token stands."""
    rng = np.random.default_rng(T + 1)
    H, V, k = 64, 512, 20
    W, h = _tensor(rng, V, H, std=0.3, dtype=dtype), _tensor(rng, T, H, dtype=dtype)
    top = rng.integers(0, V, T)
    lab = W.float()[torch.from_numpy(top).cuda()]
    h = (h.float() * 0.3 + 25.0 * lab / lab.square().sum(1, keepdim=True)).to(DT[dtype])
    z = _np(h) @ _np(W).T
    keep = z.argmax(1)
    ids = np.argsort(-z, axis=1)[:, :k]
    s = np.take_along_axis(z, ids, 1) + 0.1 * rng.normal(size=(T, k))
    s[:, 0] += 1.0
    at = np.argsort(-s, axis=1)
    assert np.all(np.take_along_axis(ids, at, 1)[:, 0] == keep)
    if order == "rising":
        at = at[:, ::-1]
    if order == "shuffled":
        at = rng.permuted(at, axis=1)
    ids = np.take_along_axis(ids, at, 1).astype(np.int32).copy()
    s = np.take_along_axis(s, at, 1).astype(np.float32).copy()
    _check(_run(h, W, ids, s, dtype, pieces), h, W, ids, s, dtype, True)
