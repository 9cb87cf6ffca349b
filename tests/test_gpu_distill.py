"""Distillation from a teacher's listed tokens on a GB300 against its fp64 definition.

Bounds, per element, from the roundings (as for the head loss):
  - an output of type bf16 is rounded once: 2^-8 of its value (2^-24 for fp32);
  - a logit is off by at most 2^-21 of the largest sum of its terms' magnitudes, which moves log p
    by twice that, and a probability by as much of itself;
  - a loss sums q (log q - log p): besides what log p is off by (with the mass of q as a factor),
    each term has some six fp32 roundings of numbers no larger than |a| + |log q| + |log p|, so
    2^-21 of the sum of q times those;
  - bf16 heads round the gradient of the logits to bf16 before the gradient products, and keep the
    softmax numerators with 11 bits in between: 2^-8 + 2^-11 of the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _tensor(rng, *shape, std=1.0, dtype="f32"):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).cuda().to(DT[dtype])


def _near(got, want, bound, name):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want)
    worst = np.unravel_index(np.argmax(off - bound), off.shape) if np.ndim(off) else ()
    assert np.all(off <= bound), (name, worst, got[worst], want[worst], np.max(off))


def run(T, H, V, r, k, dtype, form="full", n_emit=None, reduction="mean", loss_scale=1.0, pieces=0,
        weighted=False, ignored=0, grads="all", seed=0, lse=False, t_scale=1.0, lists="mixed",
        poison=False, std=None, spread=3.0, masked=None):
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(seed)
    n_emit = n_emit or V
    emit = np.sort(rng.permutation(V)[:n_emit])
    Vh = n_emit if form == "d2t" else V
    std = std or H ** -0.5
    W = _tensor(rng, Vh, H, std=std, dtype=dtype)
    w1 = _tensor(rng, V, r, std=0.3, dtype=dtype) if r else None
    w2 = _tensor(rng, r, Vh, std=0.3, dtype=dtype) if r else None
    hidden = _tensor(rng, T, H, std=2.0, dtype=dtype)
    bias = b = None
    if form == "bias":
        b = np.full(V, -1e9, np.float32)
        b[emit] = rng.normal(size=n_emit).astype(np.float32)
        bias = torch.from_numpy(b).cuda()
    d2t = torch.from_numpy(emit.astype(np.int32)).cuda() if form == "d2t" else None
    # lists of the whole vocabulary, of what the head can emit, shorter ones, empty ones
    ids = np.stack([rng.permutation(V)[:k] for _ in range(T)]).astype(np.int32)
    for t in range(T):
        if lists == "mixed" and t % 3 and k <= n_emit:
            ids[t] = emit[rng.permutation(n_emit)[:k]]
    s = np.sort(rng.normal(size=(T, k)).astype(np.float32) * spread, axis=1)[:, ::-1].copy() + 11
    if lists == "mixed":
        for t in range(0, T, 4):
            n = rng.integers(0, k + 1)
            ids[t, n:] = -1
            s[t, n:] = np.nan                     # (what an absent token brings is not read)
        for t in range(1, T, 5):
            s[t, rng.integers(0, k):] = -np.inf
    if masked is not None:                        # (some tokens of a row, or all)
        of = rng.uniform(size=(T, k)) < 0.4
        of[T // 2] = True
        s[of & np.isfinite(s)] = masked
    off = rng.permutation(T)[:ignored]
    ids[off] = -1
    prev = rng.integers(0, V, T).astype(np.int32)
    wt = rng.uniform(0, 2, T).astype(np.float32) if weighted else None
    tl = None
    if lse:
        x = np.where((ids >= 0) & np.isfinite(s), s * t_scale, -np.inf).astype(np.float64)
        with np.errstate(divide="ignore"):
            tl = np.logaddexp.reduce(x, axis=1) + rng.uniform(0, 0.5, T)
        tl = np.where(np.isfinite(tl), tl, 0.0).astype(np.float32)
    ref = [hidden.clone(), W.clone(), None if w2 is None else w2.clone()]
    if poison:
        hidden[torch.from_numpy(off).cuda()] = float("nan")
        if bias is not None:
            dead = torch.from_numpy(b <= -1e8).cuda()
            W[dead] = float("inf")
            if r:
                w2[:, dead] = float("nan")
    head = tio.Head(W, w1, w2, bias, d2t)
    cfg = tio.make_loss_config(T, H, V, r, dtype, reduction, loss_scale, pieces)
    out = tio.LossOutputs.allocate(cfg, head, d_hidden=grads != "none", d_lm_head=grads == "all",
                                   d_markov=grads != "none")
    teacher = tio.Teacher(torch.from_numpy(ids).cuda(), torch.from_numpy(s).cuda(),
                          None if tl is None else torch.from_numpy(tl).cuda(), t_scale)
    ws = tio.distill_workspace_for(cfg, head, teacher, out)
    ws.fill_(0xFF)          # (NaN and -1 wherever nothing was written)
    args = (cfg, head, teacher, hidden, torch.from_numpy(prev).cuda(), out, ws,
            None if wt is None else torch.from_numpy(wt).cuda())
    tio.distill_loss(*args)
    torch.cuda.synchronize()
    assert tio.device_status(ws) == 0
    o = to.distill_loss(_np(ref[0]), _np(ref[1]), ids, s, tl, np.float32(t_scale),
                        prev if r else None, _np(w1), _np(ref[2]), _np(bias),
                        None if d2t is None else emit, wt, reduction, loss_scale, V)
    return out, o, args


def check(out, o, dtype):
    mag = o["mag"]
    dz = mag["z"] * 2.0 ** -21 + 2.0 ** -20
    assert int(out.n_rows) == o["n_rows"]
    each = 2 * dz * max(1.0, mag["q"]) + 2.0 ** -21 * mag["loss"]
    _near(out.loss, o["loss"], each, "loss")
    if o["n_rows"]:
        share = np.sum(each) / max(1e-30, np.sum(mag["loss"]))
        _near(float(out.total), o["total"],
              mag["total"] * (share + 2.0 ** -21) + abs(o["total"]) * 2.0 ** -21
              + 2 * dz * mag["q"] * mag["total"] / max(1e-30, np.max(mag["loss"])), "total")
    q = (2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 0.0) + 4 * dz + 2.0 ** -19
    for name in ("d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        g = getattr(out, name)
        if g is not None:
            _near(g, o[name], OUT[dtype] * np.abs(o[name]) + q * mag[name] * (1 + OUT[dtype])
                  + 1e-30, name)


CASES = [
    dict(T=1, H=64, V=128, r=8, k=1), dict(T=1, H=8, V=8, r=1, k=8), dict(T=2, H=72, V=256, r=0, k=3),
    dict(T=63, H=128, V=1000, r=16, k=17), dict(T=129, H=136, V=1032, r=65, k=33),
    dict(T=257, H=200, V=2056, r=128, k=64, ignored=100), dict(T=40, H=1024, V=3000, r=256, k=256),
    dict(T=300, H=320, V=4104, r=72, k=5, ignored=300), dict(T=64, H=64, V=264, r=512, k=20),
    dict(T=60, H=64, V=1000, r=8, k=20, form="bias", n_emit=100),
    dict(T=60, H=64, V=1000, r=8, k=20, form="bias", n_emit=8),
    dict(T=150, H=96, V=5000, r=24, k=64, form="bias", n_emit=1240, ignored=30, weighted=True),
    dict(T=60, H=64, V=1000, r=8, k=40, form="d2t", n_emit=104),
    dict(T=200, H=64, V=5000, r=16, k=10, form="d2t", n_emit=2048, weighted=True, reduction="sum"),
    dict(T=130, H=128, V=2000, r=16, k=30, pieces=3), dict(T=130, H=128, V=2000, r=16, k=30, pieces=99),
    dict(T=50, H=128, V=2000, r=16, k=30, pieces=3),
    dict(T=90, H=64, V=3000, r=8, k=12, form="bias", n_emit=304, pieces=4),
    dict(T=100, H=64, V=1024, r=16, k=9, loss_scale=128.0, reduction="sum"),
    dict(T=100, H=64, V=1024, r=16, k=9, grads="frozen"),
    dict(T=100, H=64, V=1024, r=16, k=9, grads="none"),
    dict(T=100, H=64, V=1024, r=16, k=50, lse=True, t_scale=0.5),
    dict(T=100, H=64, V=1024, r=16, k=50, t_scale=2.0, spread=40.0),
    dict(T=100, H=64, V=1024, r=16, k=50, lse=True, std=3.0, weighted=True),
]



@pytest.mark.parametrize("masked", [-3.4028234e38, -1e9, -1e4])
@pytest.mark.parametrize("t_scale", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("dtype,pieces", [("f32", 0), ("f32", 3), ("bf16", 0), ("bf16", 3)])
def test_listed_tokens_masked_by_a_number(masked, t_scale, dtype, pieces):
    """Their q is 0 and their entry of the gradient Q p, not what log q - (log q - log p) leaves."""
    for T in (9, 130):
        out, o, _ = run(T, 64, 1000, 16, 20, dtype, masked=masked, t_scale=t_scale, pieces=pieces,
                        std=0.3)
        check(out, o, dtype)

@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill(case, dtype):
    out, o, _ = run(dtype=dtype, **case)
    check(out, o, dtype)


@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_carries_no_loss_is_not_read(form, dtype):
    out, o, _ = run(T=60, H=64, V=1000, r=8, k=20, form=form,
                    n_emit=None if form == "full" else 200, ignored=25, poison=True, dtype=dtype)
    check(out, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_that_agrees_with_its_teacher(dtype):
    """Listed log q equal to the head's own log p: the loss is 0, and the listed entries of the
    gradient are what the teacher's sum leaves, without the difference of two probabilities."""
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(0)
    T, H, V, k = 24, 64, 512, 512 // 2
    W, h = _tensor(rng, V, H, std=0.3, dtype=dtype), _tensor(rng, T, H, dtype=dtype)
    z = _np(h) @ _np(W).T
    ids = np.argsort(-z, axis=1)[:, :k].astype(np.int32).copy()
    s = np.take_along_axis(z, ids, 1).astype(np.float32)
    lse = np.logaddexp.reduce(z, axis=1).astype(np.float32)
    head = tio.Head(W, None, None, None, None)
    cfg = tio.make_loss_config(T, H, V, 0, dtype)
    out = tio.LossOutputs.allocate(cfg, head)
    teacher = tio.Teacher(torch.from_numpy(ids).cuda(), torch.from_numpy(s).cuda(),
                          torch.from_numpy(lse).cuda())
    ws = tio.distill_workspace_for(cfg, head, teacher, out)
    tio.distill_loss(cfg, head, teacher, h, None, out, ws)
    o = to.distill_loss(_np(h), _np(W), ids, s, lse)
    check(out, o, dtype)
    # log q and log p are each off by 2^-20 of logits up to 16
    assert float(out.loss.abs().max()) < 2.0 ** -15


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_listed_token_is_the_head_loss(dtype):
    """k = 1 with its probability normalised: cross entropy with that token as the label."""
    from dspark_block_drafter_gb300 import torch_io as tio
    out, o, args = run(T=150, H=128, V=1000, r=16, k=1, lists="full", dtype=dtype, seed=3)
    cfg, head, teacher, hidden, prev, _, _, _ = args
    ref = tio.LossOutputs.allocate(cfg, head)
    ws = tio.loss_workspace_for(cfg, head, ref)
    tio.head_loss(cfg, head, hidden, prev, teacher.ids[:, 0].contiguous(), ref, ws)
    for name in ("loss", "total", "d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        assert torch.equal(getattr(out, name), getattr(ref, name)), name


def test_bad_lists_drop_their_rows():
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(1)
    T, H, r, k = 12, 64, 8, 6
    for dtype in ("f32", "bf16"):
        V8 = 504
        W, w1 = _tensor(rng, V8, H, dtype=dtype), _tensor(rng, V8, r, dtype=dtype)
        w2, h = _tensor(rng, r, V8, dtype=dtype), _tensor(rng, T, H, std=0.1, dtype=dtype)
        ids = np.stack([rng.permutation(V8)[:k] for _ in range(T)]).astype(np.int32)
        s = rng.normal(size=(T, k)).astype(np.float32)
        prev = rng.integers(0, V8, T).astype(np.int32)
        ids[2, 3] = V8                    # a token that is none
        ids[5, 4] = ids[5, 0]             # the same token twice
        prev[7] = -1
        ids[8, 1], s[8, 1] = ids[8, 2], -np.inf      # (absent: not a second time)
        head = tio.Head(W, w1, w2, None, None)
        cfg = tio.make_loss_config(T, H, V8, r, dtype)
        out = tio.LossOutputs.allocate(cfg, head)
        teacher = tio.Teacher(torch.from_numpy(ids).cuda(), torch.from_numpy(s).cuda())
        ws = tio.distill_workspace_for(cfg, head, teacher, out)
        tio.distill_loss(cfg, head, teacher, h, torch.from_numpy(prev).cuda(), out, ws)
        assert tio.device_status(ws) == 5
        o = to.distill_loss(_np(h), _np(W), ids, s, None, 1.0, prev, _np(w1), _np(w2))
        assert o["dropped"] == 3 and o["n_rows"] == T - 3
        check(out, o, dtype)


def test_numbers_that_are_none():
    """A listed logit that is not a number, or +infinity, is told by its row's loss and gradients;
    other rows' losses keep their values."""
    out, o, args = run(T=20, H=64, V=512, r=0, k=8, lists="full", dtype="bf16")
    from dspark_block_drafter_gb300 import torch_io as tio
    cfg, head, teacher, hidden, prev, _, ws, _ = args
    want = out.loss.clone()
    teacher.logits[3, 5] = float("nan")
    teacher.logits[9, 0] = float("inf")
    tio.distill_loss(cfg, head, teacher, hidden, prev, out, ws)
    bad = torch.zeros(20, dtype=torch.bool, device="cuda")
    bad[3] = bad[9] = True
    assert torch.isnan(out.loss[bad]).all() and torch.isnan(out.total).all()
    assert torch.isnan(out.d_hidden[bad]).any(1).all()
    assert torch.equal(out.loss[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_is_the_loss_s_difference(dtype):
    """Against differences of the fp64 loss, along random directions of hidden."""
    out, o, args = run(T=6, H=64, V=256, r=8, k=12, dtype=dtype, lse=True, seed=5)
    cfg, head, teacher, hidden, prev, _, _, _ = args
    rng = np.random.default_rng(0)
    h0, g = _np(hidden), _np(out.d_hidden)

    def total(h):
        return to.distill_loss(h, _np(head.lm_head), teacher.ids.cpu().numpy(),
                               teacher.logits.cpu().numpy(), _np(teacher.lse), 1.0,
                               prev.cpu().numpy(), _np(head.markov_w1), _np(head.markov_w2))["total"]
    for _ in range(4):
        d = rng.normal(size=h0.shape)
        want = (total(h0 + 1e-4 * d) - total(h0 - 1e-4 * d)) / 2e-4
        bound = np.sum(np.abs(d) * (OUT[dtype] * np.abs(o["d_hidden"])
                                    + 2.0 ** -7 * o["mag"]["d_hidden"] * (dtype == "bf16")
                                    + 2.0 ** -14 * o["mag"]["d_hidden"])) + 1e-5
        assert abs(np.sum(d * g) - want) <= bound
