"""The head's training operators on a GB300 against their fp64 definitions.

Bounds are derived, per element, from the roundings each operator makes:
  - an output of type bf16 is rounded once: 2^-8 of its value (2^-24 for fp32);
  - bf16 heads round the gradient of the logits to bf16 before the gradient products, and
    keep the softmax numerators with 11 bits in between: 2^-8 + 2^-11 of the sum of the
    terms' magnitudes;
  - a logit is an fp32 sum: off by at most 2^-21 of the largest sum of its terms'
    magnitudes, which moves a probability by that much relatively; an fp32 sum in a
    gradient adds 2^-20 of its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import train_oracle as to

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
    if off.size == 0:
        return
    worst = np.unravel_index(np.argmax(off - bound), off.shape) if off.ndim else ()
    assert np.all(off <= bound), (name, worst, got[worst], want[worst], np.max(off))


def run_loss(T, H, V, r, dtype, form="full", n_emit=None, reduction="mean", loss_scale=1.0,
             pieces=0, weighted=False, ignored=0, grads="all", seed=0, prev_range=None,
             poison=False, labels=None, std=None):
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
    bias = None
    if form == "bias":
        b = np.full(V, -1e9, np.float32)
        b[emit] = rng.normal(size=n_emit).astype(np.float32)
        bias = torch.from_numpy(b).cuda()
    d2t = torch.from_numpy(emit.astype(np.int32)).cuda() if form == "d2t" else None
    lab = emit[rng.integers(0, n_emit, T)].astype(np.int32) if labels is None else labels
    off = rng.permutation(T)[:ignored]
    lab[off] = -1
    prev = rng.integers(0, prev_range or V, T).astype(np.int32)
    wt = rng.uniform(0, 2, T).astype(np.float32) if weighted else None
    ref = [hidden.clone(), W.clone(), None if w2 is None else w2.clone()]
    if poison:              # whatever a row without a loss or a masked row holds is not read
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
    ws = tio.loss_workspace_for(cfg, head, out)
    ws.fill_(0xFF)          # (NaN and -1 wherever nothing was written)
    args = (cfg, head, hidden, torch.from_numpy(prev).cuda(), torch.from_numpy(lab).cuda(), out,
            ws, None if wt is None else torch.from_numpy(wt).cuda())
    tio.head_loss(*args)
    torch.cuda.synchronize()
    assert tio.device_status(ws) == 0
    o = to.head_loss(_np(ref[0]), _np(ref[1]), lab, prev if r else None, _np(w1), _np(ref[2]),
                     _np(bias), None if d2t is None else emit, wt, reduction, loss_scale, V)
    return out, o, args


def check_loss(out, o, dtype):
    mag = o["mag"]
    dz = mag["z"] * 2.0 ** -21 + 2.0 ** -20
    assert int(out.n_rows) == o["n_rows"]
    _near(out.loss, o["loss"], 2 * dz + 2.0 ** -22 * np.abs(o["loss"]), "loss")
    scale = abs(o["total"]) * 2.0 ** -22 + 2 * dz * max(1.0, abs(o["total"]) / max(
        1e-30, np.abs(o["loss"]).max()))
    _near(float(out.total), o["total"], scale, "total")
    q = (2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 0.0) + 2 * dz + 2.0 ** -20
    for name in ("d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        g = getattr(out, name)
        if g is not None:
            _near(g, o[name], OUT[dtype] * np.abs(o[name]) + q * mag[name] * (1 + OUT[dtype])
                  + 1e-30, name)


def check_few_rows(out, o):
    """bf16, up to 64 rows: the products see the gradient of the logits with 16 bits, so that
    only the kept numerators' 2^-10.8 stays besides the output's own rounding."""
    mag = o["mag"]
    eps = 2.0 ** -10.7 + 2 * (mag["z"] * 2.0 ** -21 + 2.0 ** -20) + 2.0 ** -20
    for name in ("d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        g = getattr(out, name)
        if g is not None:
            _near(g, o[name], 2.0 ** -8 * np.abs(o[name]) + eps * mag[name] * (1 + 2.0 ** -8)
                  + 1e-30, name)


LOSS_CASES = [
    # one row, one tile, and past tile edges in every dimension
    dict(T=1, H=64, V=128, r=8), dict(T=1, H=8, V=8, r=1), dict(T=2, H=72, V=256, r=0),
    dict(T=127, H=128, V=1000, r=16), dict(T=129, H=136, V=1032, r=65),
    dict(T=256, H=64, V=512, r=64), dict(T=257, H=200, V=2056, r=128, ignored=100),
    dict(T=300, H=320, V=4104, r=72, ignored=299), dict(T=40, H=1024, V=3000, r=256),
    dict(T=700, H=64, V=264, r=512),
    # reduced vocabularies
    dict(T=60, H=64, V=1000, r=8, form="bias", n_emit=100),
    dict(T=60, H=64, V=1000, r=8, form="bias", n_emit=1),
    dict(T=60, H=64, V=1000, r=8, form="bias", n_emit=1000),
    dict(T=150, H=96, V=5000, r=24, form="bias", n_emit=1237, ignored=30, weighted=True),
    dict(T=60, H=64, V=1000, r=0, form="bias", n_emit=257),
    dict(T=60, H=64, V=1000, r=8, form="d2t", n_emit=104),
    dict(T=200, H=64, V=5000, r=16, form="d2t", n_emit=2048, weighted=True, reduction="sum"),
    # pieces, scales, frozen parts
    dict(T=130, H=128, V=2000, r=16, pieces=3), dict(T=130, H=128, V=2000, r=16, pieces=1000),
    dict(T=90, H=64, V=3000, r=8, form="bias", n_emit=300, pieces=4),
    dict(T=100, H=64, V=1024, r=16, loss_scale=128.0, reduction="sum"),
    dict(T=100, H=64, V=1024, r=16, grads="frozen"), dict(T=100, H=64, V=1024, r=16, grads="none"),
    dict(T=100, H=64, V=1024, r=16, grads="frozen", pieces=2),
    # every row shares one prev
    dict(T=500, H=64, V=520, r=32, prev_range=1),
    # large logits: the softmax needs its maximum
    dict(T=64, H=256, V=1024, r=16, std=4.0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LOSS_CASES, ids=lambda c: "-".join(
    f"{k}{v}" for k, v in c.items()))
def test_loss(case, dtype):
    out, o, _ = run_loss(dtype=dtype, seed=len(str(case)), **case)
    check_loss(out, o, dtype)


@pytest.mark.parametrize("pieces", [1, 3])
@pytest.mark.parametrize("T,ignored", [(1, 0), (5, 0), (64, 0), (90, 26), (128, 64)])
def test_loss_of_few_rows_rounds_only_its_outputs(T, ignored, pieces):
    out, o, _ = run_loss(T, 192, 1544, 24, "bf16", ignored=ignored, pieces=pieces, weighted=True,
                         prev_range=9)
    check_few_rows(out, o)


@pytest.mark.parametrize("pieces", [1, 3])
@pytest.mark.parametrize("T,H,V", [(1, 192, 1504), (7, 192, 1504), (100, 192, 1504),
                                   (300, 128, 4096)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_losses_keep_their_digits(dtype, T, H, V, pieces):
    """Rows whose label has nearly all the probability: losses down to 1e-9, and gradients as
    small, to the same relative precision as large ones."""
    from dspark_block_drafter_gb300 import torch_io as tio
    out, _, args = run_loss(T, H, V, 0, dtype, pieces=pieces)
    cfg, head, hidden, _, labels, _, ws, _ = args
    W, lab = _np(head.lm_head), labels.cpu().numpy()
    much = np.linspace(26, 13, T)[:, None]
    hidden.copy_(torch.from_numpy((W[lab] * much).astype(np.float32)))
    tio.head_loss(*args)
    torch.cuda.synchronize()
    o = to.head_loss(_np(hidden), W, lab, V=V)
    assert o["loss"].min() < 1e-4
    dz = o["mag"]["z"] * 2.0 ** -21 + 2.0 ** -20
    _near(out.loss, o["loss"], o["loss"] * (2 * dz + 2.0 ** -18), "loss")
    _near(float(out.total), o["total"], o["total"] * (2 * dz + 2.0 ** -18), "total")
    check_loss(out, o, dtype)
    if dtype == "bf16" and T <= 64:
        check_few_rows(out, o)


@pytest.mark.parametrize("case", [
    dict(H=33, V=1, dtype="f32"), dict(H=33, V=500, dtype="f32", form="bias", n_emit=1),
    dict(H=64, V=512, dtype="bf16", form="bias", n_emit=1)], ids=str)
@pytest.mark.parametrize("T", [1, 20, 200])
def test_loss_of_one_head_row_is_zero(case, T):
    out, _, _ = run_loss(T=T, r=8, ignored=T // 4, **case)
    assert int(out.n_rows) == T - T // 4
    for name in ("loss", "total", "d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        assert not getattr(out, name).any(), name


@pytest.mark.parametrize("case", [
    dict(T=3, H=7, V=13, r=3), dict(T=65, H=33, V=131, r=5), dict(T=97, H=129, V=1001, r=17),
    dict(T=31, H=65, V=777, r=9, form="bias", n_emit=101),
    dict(T=31, H=65, V=777, r=9, form="d2t", n_emit=101, pieces=2)], ids=str)
def test_loss_odd_sizes_f32(case):
    out, o, _ = run_loss(dtype="f32", **case)
    check_loss(out, o, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pieces", [1, 2])
def test_loss_does_not_read_what_is_masked(dtype, pieces):
    out, o, _ = run_loss(140, 128, 1504, 24, dtype, form="bias", n_emit=700, ignored=50,
                         poison=True, pieces=pieces)
    check_loss(out, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
def test_loss_of_no_rows(dtype, form):
    for grads in ("all", "none"):
        out, o, _ = run_loss(20, 64, 512, 8, dtype, form=form, n_emit=64, ignored=20,
                             grads=grads, poison=True)
        check_loss(out, o, dtype)
        assert float(out.total) == 0 and not out.loss.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_with_every_head_row_masked(dtype):
    from dspark_block_drafter_gb300 import torch_io as tio
    T, H, V = 9, 64, 256
    head = tio.Head(torch.full((V, H), float("nan"), device="cuda", dtype=DT[dtype]), None, None,
                    torch.full((V,), -1e9, device="cuda"))
    cfg = tio.make_loss_config(T, H, V, 0, dtype)
    out = tio.LossOutputs.allocate(cfg, head)
    ws = tio.loss_workspace_for(cfg, head, out)
    ws.fill_(0xFF)
    tio.head_loss(cfg, head, torch.ones(T, H, device="cuda", dtype=DT[dtype]), None,
                  torch.arange(T, device="cuda", dtype=torch.int32), out, ws)
    assert tio.device_status(ws) == 0
    assert int(out.n_rows) == 0 and float(out.total) == 0 and not out.loss.any()
    assert not out.d_hidden.any() and not out.d_lm_head.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_labels_and_prev_out_of_range(dtype):
    from dspark_block_drafter_gb300 import torch_io as tio
    out, o, args = run_loss(10, 64, 128, 8, dtype)
    cfg, head, hidden, prev, labels, out, ws, _ = args
    want = out.loss.clone()
    for t, bad in ((labels, 128), (prev, -1), (prev, 128)):
        keep = t[4].item()
        t[4] = bad
        tio.head_loss(*args)
        assert tio.device_status(ws) == 5
        assert int(out.n_rows) == 9 and out.loss[4] == 0 and not out.d_hidden[4].any()
        assert torch.equal(out.loss[:4], want[:4]) and torch.equal(out.loss[5:], want[5:])
        t[4] = keep
    labels[4] = -1
    prev[4] = -7               # a row without a loss: its prev is not looked at
    tio.head_loss(*args)
    assert tio.device_status(ws) == 0 and int(out.n_rows) == 9


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_repeats_its_bits(dtype):
    from dspark_block_drafter_gb300 import torch_io as tio
    out, _, args = run_loss(333, 128, 3016, 40, dtype, ignored=20, weighted=True, prev_range=40)
    first = [t.clone() for t in (out.loss, out.total, out.d_hidden, out.d_lm_head,
                                 out.d_markov_w1, out.d_markov_w2)]
    for _ in range(3):
        tio.head_loss(*args)
        for a, b in zip(first, (out.loss, out.total, out.d_hidden, out.d_lm_head,
                                out.d_markov_w1, out.d_markov_w2)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_pieces_agree(dtype):
    a, o, _ = run_loss(200, 128, 4000, 16, dtype, pieces=1)
    b, _, _ = run_loss(200, 128, 4000, 16, dtype, pieces=5)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.total, b.total)
    check_loss(b, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_and_norm_on_a_side_stream_and_in_a_graph(dtype):
    from dspark_block_drafter_gb300 import torch_io as tio
    out, o, args = run_loss(70, 64, 1000, 8, dtype, form="bias", n_emit=300)
    s = torch.cuda.Stream()
    for t in (out.loss, out.d_hidden, out.d_lm_head):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    tio.head_loss(*args, stream=s)
    s.synchronize()
    check_loss(out, o, dtype)
    first = out.d_lm_head.clone()
    out.d_lm_head.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tio.head_loss(*args)
    for _ in range(2):
        out.d_lm_head.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out.d_lm_head)


# ------------------------------------------------------------------ block norm
NORM_CASES = [dict(T=1, H=1), dict(T=1, H=8), dict(T=3, H=57), dict(T=2, H=256),
              dict(T=5, H=264, post=False), dict(T=17, H=1001, span=0), dict(T=17, H=1024, span=7),
              dict(T=65, H=2816, span=1), dict(T=64, H=512, span=64), dict(T=70, H=512, span=33),
              dict(T=100, H=128, span=1000), dict(T=33, H=4096, post=False, span=0),
              dict(T=9, H=8192), dict(T=9, H=8191), dict(T=6, H=640, y=False, post=False, span=0),
              dict(T=2000, H=96, span=1), dict(T=40, H=320, offset=0.0, scale=0.1)]


def run_norm(T, H, dtype, span=1, post=True, y=True, offset=1.0, scale=0.5, seed=0, up=True,
             shift=0):
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(seed)

    def make(*shape, std=1.0):
        n = int(np.prod(shape))
        flat = _tensor(rng, n + shift, std=std, dtype=dtype)   # (shift: not 16-byte aligned)
        return flat[shift:].view(*shape)

    x, w_pre = make(T, H), make(H, std=0.2)
    yy = make(T, H, std=3.0) if y else None
    w_post = make(H, std=0.2) if post else None
    gate = make((T + span - 1) // span, H) if span else None
    dh, dxo = make(T, H), make(T, H) if up else None
    cfg = tio.make_norm_config(T, H, dtype, 1e-6, scale, offset, max(1, span))
    kw = dict(gate=gate, w_post=w_post)
    ref = dict(gate=_np(gate), w_post=_np(w_post), eps=1e-6, scale=scale, offset=offset,
               span=max(1, span))
    ref["scale"] = float(np.float32(scale))
    ref["eps"] = float(np.float32(1e-6))
    xo, h = torch.empty_like(x), torch.empty_like(x)
    tio.block_norm(cfg, x, yy, w_pre, h, x_out=xo, **kw)
    out = tio.NormGrads.allocate(cfg, span > 0, post, y)
    ws = tio.norm_workspace_for(cfg)
    ws.fill_(0xFF)
    tio.block_norm_backward(cfg, x, yy, w_pre, dh, out, ws, d_x_out=dxo, **kw)
    torch.cuda.synchronize()
    oxo, oh = to.block_norm(_np(x), _np(yy), _np(w_pre), **ref)
    o = to.block_norm_backward(_np(x), _np(yy), _np(w_pre), _np(dh), _np(dxo), **ref)
    u = OUT[dtype]
    acc = 2.0 ** -19            # fp32 sums of up to 8192 terms and a reciprocal root
    xm = np.abs(_np(x)) + np.abs(oxo - _np(x))
    _near(xo, oxo, u * np.abs(oxo) + acc * xm, "x_out")
    rx = 1 / np.sqrt((oxo ** 2).mean(1, keepdims=True) + 1e-6)
    _near(h, oh, u * np.abs(oh) + acc * (xm * rx * np.abs(offset + _np(w_pre)) + np.abs(oh)),
          "h")
    for name, want in o.items():
        if name != "mag":
            _near(getattr(out, name), want, u * np.abs(want) + acc * o["mag"][name] + 1e-30, name)
    return tio, cfg, x, yy, w_pre, h, xo, kw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_block_norm(case, dtype):
    run_norm(dtype=dtype, seed=case["T"] + case["H"], **case)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block_norm_unaligned_and_without_upstream(dtype):
    run_norm(12, 512, dtype, shift=1)
    run_norm(12, 512, dtype, up=False)


# rows made of vectors of 16, 8, 4 and 2 bytes, more of them than run at once
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,span", [(1500, 520, 5), (1500, 516, 1), (1500, 514, 0),
                                      (1500, 513, 5), (700, 2100, 7), (700, 2101, 1),
                                      (350, 4098, 3), (350, 5001, 0)])
def test_block_norm_rows_of_every_vector(T, H, span, dtype):
    tio, cfg, x, y, w_pre, h, xo, kw = run_norm(T, H, dtype, span=span)
    # in place, next to values that must neither count nor change
    edge = 3
    around = [torch.full((T * H + 2 * edge,), float("nan"), dtype=x.dtype, device="cuda")
              for _ in range(2)]
    inner = [b[edge:-edge].view(T, H) for b in around]
    for b, v in zip(inner, (x, y)):
        b.copy_(v)
    tio.block_norm(cfg, inner[0], inner[1], w_pre, inner[1], x_out=inner[0], **kw)
    u = 2 * OUT[dtype] + 2.0 ** -17         # (other vectors, other orders of the sums)
    _near(inner[0], _np(xo), u * (np.abs(_np(x)) + np.abs(_np(xo))), "x_out in place")
    top = np.abs(_np(h)).max(1, keepdims=True)
    _near(inner[1], _np(h), u * (np.abs(_np(h)) + top), "h in place")
    for b in around:
        assert torch.isnan(b[:edge]).all() and torch.isnan(b[-edge:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block_norm_in_place_and_zero_rows(dtype):
    tio, cfg, x, y, w_pre, h, xo, kw = run_norm(12, 768, dtype)
    tio.block_norm(cfg, x, y, w_pre, y, x_out=x, **kw)
    assert torch.equal(x, xo) and torch.equal(y, h)
    x.zero_()
    y.zero_()
    tio.block_norm(cfg, x, y, w_pre, h, **kw)       # (no x_out)
    assert not h.any()


# ------------------------------------------------------------------ clipping
def _clip(shapes, max_norm, in_place=False, seed=0, std=1.0, shift=0):
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(seed)
    gs = [_tensor(rng, n + shift, std=std, dtype=dt)[shift:] for n, dt in shapes]
    before = [g.clone() for g in gs]
    outs = None if in_place else [torch.full_like(g, float("nan")) for g in gs]
    gl = tio.GradList(gs, outs)
    norm = torch.empty(1, device="cuda")
    ws = tio.clip_workspace_for(gl)
    ws.fill_(0xFF)
    tio.clip_grads(gl, max_norm, norm, ws)
    want_norm, want = to.clip_grads([_np(g) for g in before], float(np.float32(max_norm)))
    _near(float(norm), want_norm, 2.0 ** -20 * want_norm, "norm")
    for i, (o, w, (n, dt)) in enumerate(zip(gl.outs, want, shapes)):
        _near(o, w, (OUT[dt] + 2.0 ** -19) * np.abs(w), f"out {i}")
    if not in_place:
        for g, b in zip(gs, before):
            assert torch.equal(g, b)
    return gl, norm, before


CLIP_SHAPES = [[(1, "f32")], [(1, "bf16")], [(0, "f32"), (5, "bf16"), (0, "bf16")],
               [(8192, "f32"), (16384, "bf16"), (8193, "f32"), (16383, "bf16")],
               [(1000003, "bf16"), (77, "f32"), (300007, "f32")],
               [(3 * i + 1, "bf16" if i % 2 else "f32") for i in range(97)],
               [(64 + i, "f32") for i in range(300)]]


@pytest.mark.parametrize("shapes", CLIP_SHAPES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("max_norm", [0.0, 0.37, 1e9])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(shapes, max_norm, in_place):
    gl, norm, before = _clip(shapes, max_norm, in_place)
    if max_norm == 1e9:
        assert all(torch.equal(o, b) for o, b in zip(gl.outs, before))
    _clip(shapes, max_norm, in_place, shift=1)


def test_clip_all_zero():
    gl, norm, _ = _clip([(100, "f32"), (100, "bf16")], 1.0, std=0.0)
    assert float(norm) == 0 and not any(o.any() for o in gl.outs)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_leaves_gradients_whose_norm_is_not_finite(bad, in_place):
    from dspark_block_drafter_gb300 import torch_io as tio
    g = [torch.randn(40000, device="cuda"), torch.randn(9, device="cuda").bfloat16()]
    g[0][31234] = bad
    keep = [t.clone() for t in g]
    gl = tio.GradList(g, None if in_place else [torch.zeros_like(t) for t in g])
    norm = torch.empty(1, device="cuda")
    tio.clip_grads(gl, 1.0, norm, tio.clip_workspace_for(gl))
    assert not torch.isfinite(norm).any()
    for o, k in zip(gl.outs, keep):
        assert torch.equal(o.nan_to_num(7.0), k.nan_to_num(7.0))


def test_clip_repeats_its_bits():
    a, n, _ = _clip([(3000001, "bf16"), (200001, "f32")], 0.5)
    for _ in range(3):
        b, m, _ = _clip([(3000001, "bf16"), (200001, "f32")], 0.5)
        assert torch.equal(n, m) and all(torch.equal(x, y) for x, y in zip(a.outs, b.outs))
