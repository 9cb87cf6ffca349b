"""The operators of a head training step, as measured cases.

    head_loss            softmax cross entropy over the vocabulary of the Markov-corrected
                         logits, with the gradients of everything they are made of
    block_norm           residual add of a block's output (normalised, gated, scaled) and
                         the norm after it: the head's two inputs
    block_norm_backward  its gradients
    clip_grads           the global norm of a list of gradients, and the clipped gradients

`run` computes them in their plain form, in fp32 torch operations, or (``own`` true)
through the package's public calls.  `exact` gives the same outputs in 64 bits, by
automatic differentiation of the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_MASK = -1.0e9                 # bias of a head row the draft cannot emit
_MASK_LEVEL = -1.0e8           # a bias at or below this masks its row


# ------------------------------------------------------------------ cases
def _loss(name, T, H, V, r, dtype="bf16", form="full", n_emit=0, grads="all", ignored=0.0,
          pieces=0, weighted=False, reduction="mean"):
    return dict(name=name, op="loss", T=T, H=H, V=V, r=r, dtype=dtype, form=form,
                n_emit=n_emit or V, grads=grads, ignored=ignored, pieces=pieces,
                weighted=weighted, reduction=reduction)


def _norm(name, T, H, dtype="bf16", backward=False, gate_span=0, post=True, offset=0.0,
          scale=1.0):
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, backward=backward,
                gate_span=gate_span, post=post, offset=offset, scale=scale)


def _clip(name, shapes, max_norm, copies=1):
    return dict(name=name, op="clip", shapes=shapes, max_norm=max_norm, copies=copies)


def listed():
    return [
        # one drafted block scored by the Qwen3-8B-shaped head: the held-out loss of a
        # single sequence, bound by one read of the head
        _loss("loss_eval_one_block", 16, 4096, 151936, 256, grads="none"),
        # 32 blocks of 16 slots, the target's lm_head shared and frozen (the drafter and
        # its Markov weights train)
        _loss("loss_frozen_head_b32", 512, 4096, 151936, 256, grads="frozen", weighted=True),
        # a training batch of 256 blocks of 16 slots, every weight of the head trained
        _loss("loss_full_step", 4096, 4096, 151936, 256, ignored=0.1),
        # the Gemma-4-shaped reduced vocabulary in its bias form, 64 blocks of 1 + 6 slots
        # (slot 0 carries no label)
        _loss("loss_reduced_vocab", 448, 2816, 262144, 128, form="bias", n_emit=32768,
              ignored=1.0 / 7.0),
        # a d2t head, a ragged batch and the vocabulary in four pieces (bounded workspace)
        _loss("loss_pieces_ragged", 1001, 1024, 131072, 72, form="d2t", n_emit=64008,
              ignored=0.3, pieces=4, weighted=True, reduction="sum"),
        # the fp32 reference head
        _loss("loss_tiny_f32", 8, 256, 4096, 16, dtype="f32"),
        # one block's 16 slots before the 27B-shaped head: the decoding step
        _norm("norm_decode", 16, 5120),
        # a training batch through the last block, forward and backward
        _norm("norm_batch", 8192, 4096, gate_span=1, scale=0.5),
        _norm("norm_batch_backward", 8192, 4096, backward=True, gate_span=1, scale=0.5),
        # fp32, odd sizes, one gate row for each block of 16 tokens
        _norm("norm_odd_f32_backward", 337, 1001, dtype="f32", backward=True, gate_span=16,
              offset=1.0),
        # the gradients of the fp32 reference head
        _clip("clip_tiny", "4096x256:f32,4096x16:f32,16x4096:f32,256:f32", 0.5),
        # the gradients of the Qwen3-8B-shaped head and of a drafter layer before it
        _clip("clip_head", "151936x4096:bf16,151936x256:bf16,256x151936:bf16,"
              "12288x4096:bf16,4096x12288:bf16,4096x4096:bf16,4096:f32,4096:f32", 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _free(n, step):
    """n, moved off the one size that no case has."""
    return n + step if n == 3072 else n


def draw(rng):
    kind = rng.choice(["loss", "loss", "loss", "loss", "norm", "norm", "norm", "clip", "clip"])
    if kind == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return {k: v for k, v in _norm(
            "", _free(_log(rng, 1, 8192), 1), _free(_log(rng, 32, 5120), 1), dtype,
            backward=rng.random() < 0.6, gate_span=rng.choice([0, 1, 1, 7, 16]),
            post=rng.random() < 0.7, offset=rng.choice([0.0, 1.0]),
            scale=rng.choice([1.0, 0.5, 0.22])).items() if k != "name"}
    if kind == "clip":
        n = _log(rng, 1, 24)
        shapes = ",".join("%dx%d:%s" % (_free(_log(rng, 1, 30000), 1), _free(_log(rng, 1, 2000), 1),
                                        rng.choice(["bf16", "f32"])) for _ in range(n))
        return {k: v for k, v in _clip("", shapes, rng.choice([0.5, 1.0, 1.0e6]),
                                       rng.choice([1, 1, 3])).items() if k != "name"}
    if rng.random() < 0.2:
        dtype = "f32"
        T, H = _log(rng, 1, 256), _log(rng, 16, 512)
        V, r = _log(rng, 64, 8192), _log(rng, 1, 64)
        n_emit = max(1, V // rng.choice([2, 3, 8]))
    else:
        dtype = "bf16"
        T, H = _log(rng, 1, 4096), 8 * _log(rng, 8, 640)
        V, r = 8 * _log(rng, 16, 31040), rng.choice([0, 16, 40, 72, 128, 256])
        n_emit = max(8, V // rng.choice([2, 3, 8]) // 8 * 8)
        T = max(1, min(T, int(4096 * 4096 * 151936 / (H * V))))
    T, H, V = _free(T, 1), _free(H, 8), _free(V, 8)
    n_emit = min(V, _free(n_emit, 8))
    form = rng.choice(["full", "full", "bias", "d2t"])
    return {k: v for k, v in _loss(
        "", T, H, V, r, dtype, form, n_emit if form != "full" else 0,
        grads=rng.choice(["none", "frozen", "all", "all"]),
        ignored=rng.choice([0.0, 0.1, 0.5, 1.0 / 7.0]), pieces=rng.choice([0, 0, 1, 3]),
        weighted=rng.random() < 0.5, reduction=rng.choice(["mean", "sum"])).items()
        if k != "name"}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    """Normal values, drawn in row chunks so that no large fp32 copy is made."""
    out = torch.empty(*shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for a in range(0, flat.numel(), step):
        b = min(flat.numel(), a + step)
        flat[a:b] = torch.randn(b - a, generator=g, device="cuda") * std
    return out


def _skewed(g, n, k):
    """n indices in [0, k): a few frequent ones and a long tail, as tokens come."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (u ** 4 * k).long().clamp_(max=k - 1)


def _ignored_rows(case):
    return min(case["T"], int(round(case["T"] * case["ignored"])))


def _loss_inputs(c, seed):
    g = _gen(seed)
    T, H, V, r, dt = c["T"], c["H"], c["V"], c["r"], _DT[c["dtype"]]
    n_emit = c["n_emit"]
    emit = torch.randperm(V, generator=g, device="cuda")[:n_emit].sort().values \
        if n_emit < V else torch.arange(V, device="cuda")
    rows = n_emit if c["form"] == "d2t" else V
    s = {"lm_head": _randn(g, rows, H, std=0.02, dtype=dt)}
    s["w1"] = _randn(g, V, r, std=0.1, dtype=dt) if r else None
    s["w2"] = _randn(g, r, rows, std=0.1, dtype=dt) if r else None
    s["d2t"] = emit.int() if c["form"] == "d2t" else None
    s["bias"] = None
    if c["form"] == "bias":
        s["bias"] = torch.full((V,), _MASK, device="cuda")
        s["bias"][emit] = 0.0
    # labels the head can emit, and for the ignored rows -1 or a token it cannot emit
    pick = _skewed(g, T, n_emit)
    labels = emit[pick]
    lost = torch.randperm(T, generator=g, device="cuda")[:_ignored_rows(c)]
    labels[lost] = -1
    if n_emit < V and c["form"] != "full":
        hidden_token = torch.ones(V, dtype=torch.bool, device="cuda")
        hidden_token[emit] = False
        out = hidden_token.nonzero().flatten()
        labels[lost[::2]] = out[_skewed(g, lost[::2].numel(), out.numel())]
    s["labels"] = labels.int()
    s["prev"] = _skewed(g, T, V).int()
    # hidden states that favour their label by 0 to 16 in the logit: from a row the head
    # has not learned to one it predicts well
    h = _randn(g, T, H)
    lab = s["lm_head"][pick if c["form"] == "d2t" else emit[pick]].float()
    gain = torch.rand(T, 1, generator=g, device="cuda") * 16
    h += gain * lab / lab.square().sum(1, keepdim=True).clamp_min(1e-20)
    s["hidden"] = h.to(dt)
    s["weights"] = torch.rand(T, generator=g, device="cuda") + 0.5 if c["weighted"] else None
    return s


def _norm_inputs(c, seed):
    g = _gen(seed)
    T, H, dt = c["T"], c["H"], _DT[c["dtype"]]
    s = {"x": _randn(g, T, H, dtype=dt), "y": _randn(g, T, H, std=0.7, dtype=dt), "gate": None,
         "w_post": None, "d_h": None, "d_x_out": None}
    w = 1.0 - c["offset"]
    s["w_pre"] = (w + _randn(g, H, std=0.1)).to(dt)
    if c["post"]:
        s["w_post"] = (w + _randn(g, H, std=0.1)).to(dt)
    if c["gate_span"]:
        s["gate"] = _randn(g, (T + c["gate_span"] - 1) // c["gate_span"], H, dtype=dt)
    if c["backward"]:
        s["d_h"] = _randn(g, T, H, std=0.01, dtype=dt)
        s["d_x_out"] = _randn(g, T, H, std=0.01, dtype=dt)
    return s


def _shapes(c):
    out = []
    for part in c["shapes"].split(",") * c["copies"]:
        dims, dt = part.split(":")
        out.append(([int(d) for d in dims.split("x")], _DT[dt]))
    return out


def _clip_inputs(c, seed):
    g = _gen(seed)
    return {"grads": [_randn(g, *shape, std=0.01 * 3.0 ** (i % 3), dtype=dt)
                      for i, (shape, dt) in enumerate(_shapes(c))]}


def _inputs(case, seed):
    return {"loss": _loss_inputs, "norm": _norm_inputs, "clip": _clip_inputs}[case["op"]](
        case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s["own"] = _handles(case, s)
    return s


# ------------------------------------------------------------------ the package's calls
def _handles(c, s):
    from dspark_block_drafter_gb300 import torch_io as tio
    if c["op"] == "loss":
        head = tio.Head(s["lm_head"], s["w1"], s["w2"], s["bias"], s["d2t"])
        cfg = tio.make_loss_config(c["T"], c["H"], c["V"], c["r"], c["dtype"],
                                   reduction=c["reduction"], vocab_pieces=c["pieces"])
        out = tio.LossOutputs.allocate(cfg, head, d_hidden=c["grads"] != "none",
                                       d_lm_head=c["grads"] == "all",
                                       d_markov=c["grads"] != "none")
        return dict(tio=tio, cfg=cfg, head=head, out=out,
                    ws=tio.loss_workspace_for(cfg, head, out))
    if c["op"] == "norm":
        cfg = tio.make_norm_config(c["T"], c["H"], c["dtype"], eps=1e-6,
                                   residual_scale=c["scale"], weight_offset=c["offset"],
                                   gate_span=max(1, c["gate_span"]))
        h = dict(tio=tio, cfg=cfg)
        if c["backward"]:
            h["out"] = tio.NormGrads.allocate(cfg, gate=s["gate"] is not None,
                                              w_post=s["w_post"] is not None)
            h["ws"] = tio.norm_workspace_for(cfg)
        else:
            h["x_out"], h["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        return h
    outs = [torch.empty_like(t) for t in s["grads"]]
    grads = tio.GradList(s["grads"], outs)
    return dict(tio=tio, grads=grads, outs=outs, norm=torch.empty(1, device="cuda"),
                ws=tio.clip_workspace_for(grads))


def _run_own(s):
    c, o = s["case"], s["own"]
    tio = o["tio"]
    if c["op"] == "loss":
        out = o["out"]
        tio.head_loss(o["cfg"], o["head"], s["hidden"], s["prev"], s["labels"], out, o["ws"],
                      weights=s["weights"])
        d = {"total": out.total, "loss": out.loss}
        if c["grads"] != "none":
            d["d_hidden"] = out.d_hidden
            if c["r"]:
                d["d_markov_w1"], d["d_markov_w2"] = out.d_markov_w1, out.d_markov_w2
        if c["grads"] == "all":
            d["d_lm_head"] = out.d_lm_head
        return d
    if c["op"] == "norm" and not c["backward"]:
        tio.block_norm(o["cfg"], s["x"], s["y"], s["w_pre"], o["h"], x_out=o["x_out"],
                       gate=s["gate"], w_post=s["w_post"])
        return {"x_out": o["x_out"], "h": o["h"]}
    if c["op"] == "norm":
        out = o["out"]
        tio.block_norm_backward(o["cfg"], s["x"], s["y"], s["w_pre"], s["d_h"], out, o["ws"],
                                d_x_out=s["d_x_out"], gate=s["gate"], w_post=s["w_post"])
        d = {"d_x": out.d_x, "d_y": out.d_y, "d_w_pre": out.d_w_pre}
        if s["gate"] is not None:
            d["d_gate"] = out.d_gate
        if s["w_post"] is not None:
            d["d_w_post"] = out.d_w_post
        return d
    tio.clip_grads(o["grads"], c["max_norm"], o["norm"], o["ws"])
    return {"norm": o["norm"], "grads": o["outs"]}


# ------------------------------------------------------------------ the plain forms
def _plain_loss(s):
    c = s["case"]
    dt = _DT[c["dtype"]]
    T, V, r = c["T"], c["V"], c["r"]
    # head row of every label, -1 where the row carries no loss
    row_of = torch.full((V,), -1, dtype=torch.long, device="cuda")
    if s["d2t"] is not None:
        rows = None
        row_of[s["d2t"].long()] = torch.arange(s["d2t"].numel(), device="cuda")
    elif s["bias"] is not None:
        rows = (s["bias"] > _MASK_LEVEL).nonzero().flatten()
        row_of[rows] = torch.arange(rows.numel(), device="cuda")
    else:
        rows = None
        row_of = torch.arange(V, device="cuda")
    lab = s["labels"].long()
    target = torch.where(lab >= 0, row_of[lab.clamp_min(0)], lab)
    tok = (target >= 0).nonzero().flatten()
    target = target[tok]
    prev = s["prev"].long()[tok]
    w = torch.ones(T, device="cuda") if s["weights"] is None else s["weights"]
    w = w[tok]
    denom = w.sum() if c["reduction"] == "mean" else torch.ones((), device="cuda")
    scale = w / torch.where(denom == 0, torch.ones_like(denom), denom)

    lm = s["lm_head"] if rows is None else s["lm_head"][rows]
    lm = lm.float()
    h = s["hidden"][tok].float()
    z = h @ lm.t()
    if r:
        w2 = (s["w2"] if rows is None else s["w2"][:, rows]).float()
        e = s["w1"][prev].float()
        z += e @ w2
    if s["bias"] is not None:
        z += s["bias"][rows]
    m = z.max(dim=1, keepdim=True).values
    at = z.gather(1, target[:, None])
    z = z.sub_(m).exp_()
    total = z.sum(dim=1, keepdim=True)
    nll = (total.log() + m - at)[:, 0]
    loss = torch.zeros(T, device="cuda")
    loss[tok] = nll
    d = {"total": (scale * nll).sum().reshape(1), "loss": loss}
    if c["grads"] == "none":
        return d
    z.mul_(scale[:, None] / total)
    z[torch.arange(tok.numel(), device="cuda"), target] -= scale
    dh = torch.zeros(T, c["H"], device="cuda")
    dh[tok] = z @ lm
    d["d_hidden"] = dh.to(dt)
    if r:
        d1 = torch.zeros(V, r, device="cuda")
        d1.index_add_(0, prev, z @ w2.t())
        d["d_markov_w1"] = d1.to(dt)
        d2 = e.t() @ z
        if rows is not None:
            d2 = torch.zeros(r, V, device="cuda").index_copy_(1, rows, d2)
        d["d_markov_w2"] = d2.to(dt)
    if c["grads"] == "all":
        dl = z.t() @ h
        if rows is not None:
            dl = torch.zeros(V, c["H"], device="cuda").index_copy_(0, rows, dl)
        d["d_lm_head"] = dl.to(dt)
    return d


def _gate_rows(s, c):
    if s["gate"] is None:
        return 1.0
    span = c["gate_span"]
    return s["gate"].float().repeat_interleave(span, dim=0)[:c["T"]]


def _plain_norm(s):
    c = s["case"]
    dt, eps, off, scale = _DT[c["dtype"]], 1e-6, c["offset"], c["scale"]
    x, y = s["x"].float(), s["y"].float()
    g = _gate_rows(s, c)
    w_pre = s["w_pre"].float() + off
    if s["w_post"] is not None:
        w_post = s["w_post"].float() + off
        ry = torch.rsqrt((y * y).mean(1, keepdim=True) + eps)
        yn = y * ry
        u = yn * w_post
    else:
        u = y
    xo = x + scale * (g * u)
    rx = torch.rsqrt((xo * xo).mean(1, keepdim=True) + eps)
    xn = xo * rx
    if not c["backward"]:
        return {"x_out": xo.to(dt), "h": (xn * w_pre).to(dt)}
    dh = s["d_h"].float()
    dn = dh * w_pre
    dxo = s["d_x_out"].float() + rx * (dn - xn * (dn * xn).mean(1, keepdim=True))
    d = {"d_x": dxo.to(dt), "d_w_pre": (dh * xn).sum(0).to(dt)}
    du = scale * (g * dxo)
    if s["gate"] is not None:
        span, n = c["gate_span"], s["gate"].shape[0]
        dg = scale * dxo * u
        if span > 1:
            dg = torch.cat([dg, dg.new_zeros(n * span - c["T"], c["H"])])
            dg = dg.view(n, span, c["H"]).sum(1)
        d["d_gate"] = dg.to(dt)
    if s["w_post"] is None:
        d["d_y"] = du.to(dt)
    else:
        d["d_w_post"] = (du * yn).sum(0).to(dt)
        dv = du * w_post
        d["d_y"] = (ry * (dv - yn * (dv * yn).mean(1, keepdim=True))).to(dt)
    return d


def _plain_clip(s):
    c = s["case"]
    total = torch.zeros((), device="cuda")
    for t in s["grads"]:
        f = t.float()
        total = total + (f * f).sum()
    norm = total.sqrt()
    coef = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


def run(state):
    if own:
        return _run_own(state)
    return {"loss": _plain_loss, "norm": _plain_norm, "clip": _plain_clip}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass needs
def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(math.prod(sh) * (4 if dt == torch.float32 else 2) for sh, dt in _shapes(c))
        el = sum(math.prod(sh) for sh, _ in _shapes(c))
        return {"bytes": 2 * n + 4, "flops": 3 * el}
    e, T, H = _size(c["dtype"]), c["T"], c["H"]
    if c["op"] == "norm":
        gate = (T + c["gate_span"] - 1) // c["gate_span"] * H if c["gate_span"] else 0
        w = H * (2 if c["post"] else 1)
        if not c["backward"]:
            return {"bytes": e * (4 * T * H + gate + w), "flops": 12 * T * H}
        return {"bytes": e * (6 * T * H + 2 * gate + 2 * w), "flops": 36 * T * H}
    V, r, Ve = c["V"], c["r"], c["n_emit"]
    Tv = T - _ignored_rows(c)
    rows = Ve if c["form"] == "d2t" else V
    b = Tv * (H + r) * e + Ve * (H + r) * e + 12 * T + 4
    b += 4 * T if c["weighted"] else 0
    b += 4 * rows if c["form"] != "full" else 0
    f = 2 * Tv * Ve * (H + r)
    if c["grads"] != "none":
        b += T * H * e + (V * r + r * rows) * e
        f += 2 * Tv * Ve * (H + 2 * r)
    if c["grads"] == "all":
        b += rows * H * e
        f += 2 * Tv * Ve * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ 64 bits
def _exact_loss(c, seed):
    if work(c)["flops"] > 5e12:
        return None                # more than about 20 seconds of fp64 products
    s = _loss_inputs(c, seed)
    D = torch.float64
    want = c["grads"] != "none"
    h = s["hidden"].to(D).requires_grad_(want)
    lm = s["lm_head"].to(D).requires_grad_(c["grads"] == "all")
    with torch.enable_grad():
        z = torch.matmul(h, lm.transpose(0, 1))
        if c["r"]:
            w1 = s["w1"].to(D).requires_grad_(want)
            w2 = s["w2"].to(D).requires_grad_(want)
            z = z + torch.matmul(torch.nn.functional.embedding(s["prev"].long(), w1), w2)
        if s["bias"] is not None:
            z = torch.where(s["bias"] > _MASK_LEVEL, z + s["bias"].to(D),
                            torch.full((), float("-inf"), dtype=D, device="cuda"))
        ok = s["labels"] >= 0
        if s["d2t"] is not None:
            at = torch.searchsorted(s["d2t"], s["labels"]).clamp(max=s["d2t"].numel() - 1)
            ok = ok & (s["d2t"][at] == s["labels"])
        else:
            at = s["labels"].long().clamp_min(0)
            if s["bias"] is not None:
                ok = ok & (s["bias"][at] > _MASK_LEVEL)
        at = torch.where(ok, at, torch.zeros_like(at))
        nll = torch.logsumexp(z, dim=1) - torch.gather(z, 1, at.long()[:, None])[:, 0]
        nll = torch.where(ok, nll, torch.zeros_like(nll))
        w = ok.to(D) if s["weights"] is None else s["weights"].to(D) * ok
        total = (w * nll).sum()
        if c["reduction"] == "mean" and bool(ok.any()):
            total = total / w.sum()
    d = {"total": total.detach().reshape(1), "loss": nll.detach()}
    if not want:
        return d
    total.backward()
    d["d_hidden"] = h.grad
    if c["r"]:
        d["d_markov_w1"], d["d_markov_w2"] = w1.grad, w2.grad
    if c["grads"] == "all":
        d["d_lm_head"] = lm.grad
    return d


def _exact_norm(c, seed):
    s = _norm_inputs(c, seed)
    D = torch.float64
    t = {k: v.to(D).requires_grad_(c["backward"]) if v is not None else None
         for k, v in s.items() if not k.startswith("d_")}

    def rms(a, w):
        return a / (a.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (c["offset"] + w)

    with torch.enable_grad():
        u = t["y"] if t["w_post"] is None else rms(t["y"], t["w_post"])
        if t["gate"] is not None:
            rows = torch.arange(c["T"], device="cuda") // c["gate_span"]
            u = u * t["gate"][rows]
        xo = t["x"] + c["scale"] * u
        h = rms(xo, t["w_pre"])
    if not c["backward"]:
        return {"x_out": xo, "h": h}
    torch.autograd.backward([xo, h], [s["d_x_out"].to(D), s["d_h"].to(D)])
    d = {"d_x": t["x"].grad, "d_w_pre": t["w_pre"].grad}
    if t["gate"] is not None:
        d["d_gate"] = t["gate"].grad
    d["d_y"] = t["y"].grad
    if t["w_post"] is not None:
        d["d_w_post"] = t["w_post"].grad
    return d


def _exact_clip(c, seed):
    s = _clip_inputs(c, seed)
    norm = torch.stack([t.to(torch.float64).pow(2).sum() for t in s["grads"]]).sum().sqrt()
    factor = min(1.0, c["max_norm"] / (norm.item() + 1e-6))
    return {"norm": norm.reshape(1), "grads": [t.to(torch.float64) * factor for t in s["grads"]]}


def exact(case, seed):
    return {"loss": _exact_loss, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](case, seed)
