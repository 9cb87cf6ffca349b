"""What a drafter learns from and is verified against, as measured cases.

    sample          a token of every row of the target's logits: temperature, top-k, top-p,
                    min-p, and one given uniform number
    top_logits      the k largest logits of every row, and its log-sum-exp
    distill_loss    the divergence of the Markov-corrected head from a teacher's listed
                    tokens, with the gradients of everything its logits are made of
    embed           rows of the embedding table, scaled
    embed_backward  the table's gradient

`run` computes them in their plain form, in elementary torch operations, or (``own`` true)
through the package's public calls.  `exact` gives the same outputs in 64 bits, written
from the definitions once more.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_D = torch.float64
_INF = float("inf")


# ------------------------------------------------------------------ cases
def _sample(name, T, V, dtype="f32", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
            mixed=False, pad=0):
    return dict(name=name, op="sample", T=T, V=V, dtype=dtype, temperature=temperature,
                top_k=top_k, top_p=top_p, min_p=min_p, mixed=mixed, pad=pad)


def _top(name, T, V, k, dtype="f32", pad=0):
    return dict(name=name, op="top", T=T, V=V, k=k, dtype=dtype, pad=pad)


def _distill(name, T, H, V, r, k, dtype="bf16", form="full", n_emit=0, grads="all",
             ignored=0.0, pieces=0, weighted=False, reduction="mean", lse=False, scale=1.0):
    return dict(name=name, op="distill", T=T, H=H, V=V, r=r, k=k, dtype=dtype, form=form,
                n_emit=n_emit or V, grads=grads, ignored=ignored, pieces=pieces,
                weighted=weighted, reduction=reduction, lse=lse, scale=scale)


def _embed(name, T, V, H, dtype="bf16", scale=1.0, backward=False, add=False, ignored=0.0):
    return dict(name=name, op="embed", T=T, V=V, H=H, dtype=dtype, scale=scale,
                backward=backward, add=add, ignored=ignored)


def listed():
    return [
        # one block of 16 slots and its bonus token, verified against sampled tokens: the
        # smallest serving step
        _sample("sample_one_block", 17, 151936, temperature=0.7, top_k=20, top_p=0.8),
        # 32 such blocks of requests that each bring their own settings, greedy ones among them
        _sample("sample_mixed_b32", 544, 151936, "bf16", mixed=True),
        # a batch of rollouts from the nucleus, over logits in rows of padded length
        _sample("sample_nucleus", 2048, 151936, top_p=0.95, pad=64),
        # the candidates of one block
        _top("top_one_block", 16, 151936, 8),
        # the target's logits over a training batch, as the teacher's list
        _top("top_teacher_batch", 4096, 151936, 64, "bf16"),
        # the fp32 reference head
        _distill("distill_tiny_f32", 8, 256, 4096, 16, 8, dtype="f32"),
        # a d2t head, a ragged batch, the vocabulary in four pieces, the teacher's own sums
        _distill("distill_pieces_ragged", 1001, 1024, 131072, 72, 17, form="d2t", n_emit=64008,
                 ignored=0.3, pieces=4, weighted=True, reduction="sum", lse=True),
        # 128 blocks of 16 slots, every weight of the head trained, 64 listed tokens a slot
        _distill("distill_full_step", 2048, 4096, 151936, 256, 64, ignored=0.1),
        # the input rows of one block: the decoding step
        _embed("embed_one_block", 16, 151936, 4096),
        # those of a training batch
        _embed("embed_batch", 16384, 151936, 4096, scale=64.0, ignored=0.1),
        # and the gradient of the whole table
        _embed("embed_grad_batch", 16384, 151936, 4096, scale=64.0, backward=True, ignored=0.1),
        # odd sizes in fp32, onto the gradient of a tied head
        _embed("embed_grad_tied_f32", 4999, 32003, 1001, "f32", backward=True, add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "top", "top", "distill", "distill", "distill",
                     "embed", "embed"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "sample":
        V = _log(rng, 16, 262144)
        T = max(1, min(_log(rng, 1, 4096), 2048 * 151936 // V))
        c = _sample("", T, V, dtype, temperature=rng.choice([0.0, 0.6, 1.0, 1.0, 1.5]),
                    top_k=rng.choice([0, 0, 1, 20, 50, 1000]),
                    top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.4,
                    pad=rng.choice([0, 0, 1, 64]))
    elif op == "top":
        V = _log(rng, 16, 262144)
        T = max(1, min(_log(rng, 1, 4096), 2048 * 151936 // V))
        c = _top("", T, V, min(V, rng.choice([1, 2, 8, 33, 64, 256])), dtype,
                 rng.choice([0, 0, 1, 64]))
    elif op == "embed":
        c = _embed("", _log(rng, 1, 16384), _log(rng, 64, 151936), _log(rng, 8, 4096), dtype,
                   scale=rng.choice([1.0, 1.0, 0.5, 53.25]), backward=rng.random() < 0.7,
                   add=rng.random() < 0.4, ignored=rng.choice([0.0, 0.0, 0.1, 0.5]))
    else:
        if rng.random() < 0.3:
            T, H = _log(rng, 1, 256), _log(rng, 16, 512)
            V, r = _log(rng, 64, 8192), _log(rng, 1, 64)
            dtype, n_emit = "f32", max(1, V // rng.choice([2, 3, 8]))
        else:
            T, H = _log(rng, 1, 2048), 8 * _log(rng, 8, 640)
            V, r = 8 * _log(rng, 16, 31040), rng.choice([0, 16, 40, 72, 128, 256])
            dtype, n_emit = "bf16", max(8, V // rng.choice([2, 3, 8]) // 8 * 8)
            T = max(1, min(T, 2048 * 4096 * 151936 // (H * V)))
        form = rng.choice(["full", "full", "bias", "d2t"])
        n_emit = n_emit if form != "full" else V
        c = _distill("", T, H, V, r, min(rng.choice([1, 4, 8, 20, 64]), n_emit), dtype, form,
                     n_emit, grads=rng.choice(["none", "frozen", "all", "all"]),
                     ignored=rng.choice([0.0, 0.1, 0.5]), pieces=rng.choice([0, 0, 1, 3]),
                     weighted=rng.random() < 0.5, reduction=rng.choice(["mean", "sum"]),
                     lse=rng.random() < 0.4, scale=rng.choice([1.0, 1.0, 0.5]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _skewed(g, n, k):
    """n indices in [0, k): a few frequent ones and a long tail, as tokens come."""
    u = torch.rand(n, generator=g, device="cuda", dtype=_D)
    return (u ** 4 * k).long().clamp_(max=k - 1)


def _pick(g, n, values, dtype=torch.float32):
    at = torch.randint(len(values), (n,), generator=g, device="cuda")
    return torch.tensor(values, dtype=dtype, device="cuda")[at]


def _target_logits(g, T, V, pad, dtype):
    """Rows whose probabilities fall as a power of their rank, from rather flat ones to ones
    that have all but decided."""
    z = _rand(g, T, V + pad).mul_(V).add_(1.0).log_()
    z.mul_(_rand(g, T, 1).mul_(-1.5).sub_(0.7))
    z.add_(_randn(g, T, V + pad, std=0.5)).add_(18.0)
    return z.to(dtype)[:, :V]


def _sample_inputs(c, seed):
    g = _gen(seed)
    T = c["T"]
    s = {"logits": _target_logits(g, T, c["V"], c["pad"], _DT[c["dtype"]])}
    s["uniform"] = _rand(g, T)
    s["temperature"] = s["top_k"] = s["top_p"] = s["min_p"] = None
    if c["mixed"]:
        s["temperature"] = _pick(g, T, [0.0, 0.6, 0.8, 1.0, 1.3])
        s["top_k"] = _pick(g, T, [0, 20, 50, 200], torch.int32)
        s["top_p"] = _pick(g, T, [1.0, 0.9, 0.95])
        s["min_p"] = _pick(g, T, [0.0, 0.0, 0.05])
    return s


def _top_inputs(c, seed):
    return {"logits": _target_logits(_gen(seed), c["T"], c["V"], c["pad"], _DT[c["dtype"]])}


def _distill_inputs(c, seed):
    g = _gen(seed)
    T, H, V, r, k, dt = c["T"], c["H"], c["V"], c["r"], c["k"], _DT[c["dtype"]]
    n = c["n_emit"]
    emit = torch.arange(V, device="cuda")
    if n < V:
        emit = torch.randperm(V, generator=g, device="cuda")[:n].sort().values
    rows = n if c["form"] == "d2t" else V
    s = {"lm_head": _randn(g, rows, H, std=0.02, dtype=dt)}
    s["w1"] = _randn(g, V, r, std=0.1, dtype=dt) if r else None
    s["w2"] = _randn(g, r, rows, std=0.1, dtype=dt) if r else None
    s["d2t"] = emit.int() if c["form"] == "d2t" else None
    s["bias"] = None
    if c["form"] == "bias":
        s["bias"] = torch.full((V,), -1.0e9, device="cuda")
        s["bias"][emit] = 0.0
    # k different tokens a row, of the whole vocabulary (an eighth of the rows) or of those that
    # the head can emit; the last ones of some rows are missing, and all of those without a loss
    first, step = _skewed(g, T, n), (_rand(g, T) * (n // k)).long().clamp_(min=1)
    at = (first[:, None] + step[:, None] * torch.arange(k, device="cuda")) % n
    ids = emit[at]
    anywhere = _rand(g, T) < 0.125
    ids[anywhere] = at[anywhere]
    length = torch.where(_rand(g, T) < 0.2, (_rand(g, T) * k).long() + 1, k)
    length[_rand(g, T) < c["ignored"]] = 0
    ids[torch.arange(k, device="cuda") >= length[:, None]] = -1
    s["ids"] = ids.int()
    # the teacher's logits, falling; its own sum over the whole vocabulary is a little larger
    fall = _rand(g, T, k).log_().mul_(-0.6).cumsum(1)
    s["teacher"] = 20.0 - fall
    s["teacher_lse"] = None
    if c["lse"]:
        s["teacher_lse"] = (s["teacher"] * c["scale"]).logsumexp(1) + 0.1 * _rand(g, T)
    # hidden states that favour the first token by 0 to 10 in the logit
    h = _randn(g, T, H)
    lab = s["lm_head"][at[:, 0] if c["form"] == "d2t" else emit[at[:, 0]]].float()
    h += _rand(g, T, 1) * 10.0 * lab / lab.square().sum(1, keepdim=True).clamp_min(1e-20)
    s["hidden"] = h.to(dt)
    s["prev"] = _skewed(g, T, V).int()
    s["weights"] = _rand(g, T) + 0.5 if c["weighted"] else None
    return s


def _embed_inputs(c, seed):
    g = _gen(seed)
    T, V, H, dt = c["T"], c["V"], c["H"], _DT[c["dtype"]]
    s = {"ids": _skewed(g, T, V).int()}
    s["ids"][_rand(g, T) < c["ignored"]] = -1
    if not c["backward"]:
        s["table"] = _randn(g, V, H, std=0.02, dtype=dt)
        return s
    s["d_out"] = _randn(g, T, H, std=0.01, dtype=dt)
    s["add"] = _randn(g, V, H, std=0.01, dtype=dt) if c["add"] else None
    return s


def _inputs(case, seed):
    return {"sample": _sample_inputs, "top": _top_inputs, "distill": _distill_inputs,
            "embed": _embed_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s["own"] = _handles(case, s)
    return s


# ------------------------------------------------------------------ the package's calls
def _handles(c, s):
    from dspark_block_drafter_gb300 import torch_io as tio
    T, i32, f32 = c["T"], dict(dtype=torch.int32, device="cuda"), dict(device="cuda")
    if c["op"] == "sample":
        cfg = tio.make_sample_config(T, c["V"], c["dtype"], temperature=c["temperature"],
                                     top_k=c["top_k"], top_p=c["top_p"], min_p=c["min_p"])
        return dict(tio=tio, cfg=cfg, tokens=torch.empty(T, **i32), logp=torch.empty(T, **f32))
    if c["op"] == "top":
        return dict(tio=tio, ids=torch.empty(T, c["k"], **i32),
                    values=torch.empty(T, c["k"], **f32), lse=torch.empty(T, **f32))
    if c["op"] == "embed":
        cfg = tio.make_embed_config(T, c["V"], c["H"], c["dtype"], scale=c["scale"])
        shape = (c["V"] if c["backward"] else T, c["H"])
        out = torch.empty(shape, dtype=_DT[c["dtype"]], device="cuda")
        return dict(tio=tio, cfg=cfg, out=out,
                    ws=tio.embed_workspace_for(cfg) if c["backward"] else None)
    head = tio.Head(s["lm_head"], s["w1"], s["w2"], s["bias"], s["d2t"])
    cfg = tio.make_loss_config(T, c["H"], c["V"], c["r"], c["dtype"], reduction=c["reduction"],
                               vocab_pieces=c["pieces"])
    teacher = tio.Teacher(s["ids"], s["teacher"], lse=s["teacher_lse"], scale=c["scale"])
    out = tio.LossOutputs.allocate(cfg, head, d_hidden=c["grads"] != "none",
                                   d_lm_head=c["grads"] == "all", d_markov=c["grads"] != "none")
    return dict(tio=tio, cfg=cfg, head=head, teacher=teacher, out=out,
                ws=tio.distill_workspace_for(cfg, head, teacher, out))


def _run_own(s):
    c, o = s["case"], s["own"]
    tio = o["tio"]
    if c["op"] == "sample":
        tio.sample(o["cfg"], s["logits"], s["uniform"], o["tokens"], logp=o["logp"],
                   temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"])
        return {"tokens": o["tokens"], "logp": o["logp"]}
    if c["op"] == "top":
        tio.top_logits(s["logits"], o["ids"], o["values"], lse=o["lse"])
        return {"ids": o["ids"], "values": o["values"], "lse": o["lse"]}
    if c["op"] == "embed":
        if c["backward"]:
            tio.embed_backward(o["cfg"], s["ids"], s["d_out"], o["out"], o["ws"], add=s["add"])
            return {"d_table": o["out"]}
        tio.embed(o["cfg"], s["table"], s["ids"], o["out"])
        return {"out": o["out"]}
    out = o["out"]
    tio.distill_loss(o["cfg"], o["head"], o["teacher"], s["hidden"], s["prev"], out, o["ws"],
                     weights=s["weights"])
    d = {"total": out.total, "loss": out.loss}
    if c["grads"] != "none":
        d["d_hidden"] = out.d_hidden
        if c["r"]:
            d["d_markov_w1"], d["d_markov_w2"] = out.d_markov_w1, out.d_markov_w2
    if c["grads"] == "all":
        d["d_lm_head"] = out.d_lm_head
    return d


# ------------------------------------------------------------------ the plain forms
def _plain_sample(s):
    """The draw is a border in a long sum, so the weights are held in 64 bits."""
    c = s["case"]
    T, V = c["T"], c["V"]

    def each(name, dtype):
        if s[name] is not None:
            return s[name].to(dtype)[:, None]
        return torch.full((T, 1), c[name], dtype=torch.float32, device="cuda").to(dtype)

    tau, top_p, min_p = each("temperature", _D), each("top_p", _D), each("min_p", _D)
    top_k = each("top_k", torch.long)
    greedy = tau <= 0
    z, order = s["logits"].float().sort(dim=1, descending=True, stable=True)
    w = ((z.to(_D) - z[:, :1].to(_D)) / torch.where(greedy, torch.ones_like(tau), tau)).exp_()
    rank = torch.arange(V, device="cuda")
    keep = (rank < torch.where(top_k > 0, top_k, V)) & ((rank == 0) | ~greedy)
    w = torch.where(keep, w, torch.zeros((), dtype=_D, device="cuda"))
    below = w.cumsum(1) - w
    mass = below[:, -1:] + w[:, -1:]
    keep &= (rank == 0) | (top_p >= 1) | (below < top_p * mass)
    keep &= w >= min_p
    w = torch.where(keep, w, torch.zeros((), dtype=_D, device="cuda"))
    by_id = torch.zeros_like(w).scatter_(1, order, w)
    cum = by_id.cumsum(1)
    total = cum[:, -1:]
    at = (cum <= s["uniform"].to(_D)[:, None] * total).sum(1, keepdim=True).clamp_(max=V - 1)
    logp = (by_id.gather(1, at) / total).log()
    return {"tokens": at[:, 0].int(), "logp": logp[:, 0].float()}


def _plain_top(s):
    k = s["case"]["k"]
    z, order = s["logits"].float().sort(dim=1, descending=True, stable=True)
    m = z[:, :1]
    # (a sum of many small terms, kept in 64 bits)
    lse = m[:, 0] + (z - m).exp_().sum(1, dtype=_D).log().float()
    return {"ids": order[:, :k].int(), "values": z[:, :k].contiguous(), "lse": lse}


def _plain_distill(s):
    c = s["case"]
    dt, T, V, r = _DT[c["dtype"]], c["T"], c["V"], c["r"]
    row_of = torch.arange(V, device="cuda")
    rows = None
    if s["d2t"] is not None:
        row_of = torch.full((V,), -1, dtype=torch.long, device="cuda")
        row_of[s["d2t"].long()] = torch.arange(s["d2t"].numel(), device="cuda")
    elif s["bias"] is not None:
        rows = (s["bias"] > -1.0e8).nonzero().flatten()
        row_of = torch.full((V,), -1, dtype=torch.long, device="cuda")
        row_of[rows] = torch.arange(rows.numel(), device="cuda")
    ids = s["ids"].long()
    col = torch.where(ids >= 0, row_of[ids.clamp_min(0)], ids)
    tok = (col >= 0).any(1).nonzero().flatten()
    col = col[tok]
    on = col >= 0
    col = col.clamp_min(0)
    a = torch.where(on, s["teacher"][tok] * c["scale"], -_INF)
    if s["teacher_lse"] is not None:
        a = a - s["teacher_lse"][tok][:, None]
        q = a.exp()
    else:
        a = a - a.max(1, keepdim=True).values
        a = a - a.exp().sum(1, keepdim=True).log()
        q = a.exp()
    Q = q.sum(1, keepdim=True)
    prev = s["prev"].long()[tok]
    w = torch.ones(T, device="cuda") if s["weights"] is None else s["weights"]
    w = w[tok]
    denom = w.sum() if c["reduction"] == "mean" else torch.ones((), device="cuda")
    scale = w / torch.where(denom == 0, torch.ones_like(denom), denom)

    lm = (s["lm_head"] if rows is None else s["lm_head"][rows]).float()
    h = s["hidden"][tok].float()
    z = h @ lm.t()
    if r:
        w2 = (s["w2"] if rows is None else s["w2"][:, rows]).float()
        e = s["w1"][prev].float()
        z += e @ w2
    if s["bias"] is not None:
        z += s["bias"][rows]
    m = z.max(dim=1, keepdim=True).values
    at = z.gather(1, col)
    z = z.sub_(m).exp_()
    total = z.sum(dim=1, keepdim=True)
    lse = total.log() + m
    kl = torch.where(q > 0, q * (a - (at - lse)), torch.zeros_like(q)).sum(1)
    loss = torch.zeros(T, device="cuda")
    loss[tok] = kl
    d = {"total": (scale * kl).sum().reshape(1), "loss": loss}
    if c["grads"] == "none":
        return d
    z.mul_(Q * scale[:, None] / total)
    z.scatter_add_(1, col, -q * scale[:, None])
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


def _plain_embed(s):
    c = s["case"]
    dt, ids = _DT[c["dtype"]], s["ids"].long()
    if not c["backward"]:
        rows = s["table"][ids.clamp_min(0)].float() * c["scale"]
        return {"out": torch.where(ids[:, None] >= 0, rows, torch.zeros_like(rows)).to(dt)}
    d = torch.zeros(c["V"], c["H"], device="cuda") if s["add"] is None else s["add"].float()
    if s["add"] is not None and c["dtype"] == "f32":
        d = d.clone()
    on = ids >= 0
    d.index_add_(0, ids[on], s["d_out"][on].float() * c["scale"])
    return {"d_table": d.to(dt)}


def run(state):
    if own:
        return _run_own(state)
    return {"sample": _plain_sample, "top": _plain_top, "distill": _plain_distill,
            "embed": _plain_embed}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    T, V = c["T"], c["V"]
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "sample":
        # (an exponential as one operation)
        return {"bytes": T * V * e + T * (28 if c["mixed"] else 12), "flops": 3 * T * V}
    if c["op"] == "top":
        return {"bytes": T * V * e + T * (8 * c["k"] + 4), "flops": 3 * T * V}
    H = c["H"]
    if c["op"] == "embed":
        live = T - int(round(T * c["ignored"]))
        if not c["backward"]:
            return {"bytes": e * H * (T + min(live, V)) + 4 * T, "flops": live * H}
        return {"bytes": e * H * (live + V * (2 if c["add"] else 1)) + 4 * T,
                "flops": 2 * live * H}
    r, Ve, k = c["r"], c["n_emit"], c["k"]
    Tv = T - int(round(T * c["ignored"]))
    rows = Ve if c["form"] == "d2t" else V
    b = Tv * (H + r) * e + Ve * (H + r) * e + T * (8 * k + 12) + 4
    b += 4 * T * (int(c["weighted"]) + int(c["lse"]))
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
def _exact_sample(c, seed):
    s = _sample_inputs(c, seed)
    T, V = c["T"], c["V"]
    tokens, logps = [], []
    idx = torch.arange(V, device="cuda")
    for t in range(T):
        z = s["logits"][t].to(_D)

        def of(name):
            # (the settings are 32-bit numbers)
            v = torch.tensor(c[name], dtype=torch.float32) if s[name] is None else s[name][t]
            return float(v)

        tau, k, p, m = of("temperature"), int(of("top_k")), of("top_p"), of("min_p")
        if tau <= 0:
            best = z == z.max()
            tokens.append(torch.where(best, idx, V).min())
            logps.append(torch.zeros((), dtype=_D, device="cuda"))
            continue
        x = torch.softmax(z / tau, 0)
        order = torch.argsort(-z, stable=True)
        if 0 < k < V:
            order = order[:k]
        y = x[order] / x[order].sum()
        if p < 1:
            n = int((torch.cumsum(y, 0) - y < p).sum())
            order, y = order[:max(1, n)], y[:max(1, n)]
        order = order[y / y[0] >= m]
        ids = torch.sort(order).values
        y = x[ids] / x[ids].sum()
        j = torch.searchsorted(torch.cumsum(y, 0), s["uniform"][t].to(_D), right=True)
        j = j.clamp(max=ids.numel() - 1)
        tokens.append(ids[j])
        logps.append(torch.log(y[j]))
    return {"tokens": torch.stack(tokens).int(), "logp": torch.stack(logps)}


def _exact_top(c, seed):
    z = _top_inputs(c, seed)["logits"]
    ids, values = [], []
    for t in range(0, c["T"], 256):
        y = z[t:t + 256].to(_D)
        at = torch.argsort(y, dim=1, descending=True, stable=True)[:, :c["k"]]
        ids.append(at.int())
        values.append(torch.gather(y, 1, at))
    lse = torch.cat([torch.logsumexp(z[t:t + 256].to(_D), 1) for t in range(0, c["T"], 256)])
    return {"ids": torch.cat(ids), "values": torch.cat(values), "lse": lse}


def _exact_distill(c, seed):
    if work(c)["flops"] > 5e12:
        return None                # more than about 20 seconds of fp64 products
    s = _distill_inputs(c, seed)
    want = c["grads"] != "none"
    h = s["hidden"].to(_D).requires_grad_(want)
    lm = s["lm_head"].to(_D).requires_grad_(c["grads"] == "all")
    with torch.enable_grad():
        z = torch.matmul(h, lm.transpose(0, 1))
        if c["r"]:
            w1 = s["w1"].to(_D).requires_grad_(want)
            w2 = s["w2"].to(_D).requires_grad_(want)
            z = z + torch.matmul(torch.nn.functional.embedding(s["prev"].long(), w1), w2)
        ids = s["ids"]
        ok = ids >= 0
        if s["d2t"] is not None:
            at = torch.searchsorted(s["d2t"], ids).clamp(max=s["d2t"].numel() - 1)
            ok = ok & (s["d2t"][at] == ids)
        else:
            at = ids.long().clamp_min(0)
            if s["bias"] is not None:
                ok = ok & (s["bias"][at] > -1.0e8)
                z = torch.where(s["bias"] > -1.0e8, z + s["bias"].to(_D), -_INF)
        at = torch.where(ok, at, torch.zeros_like(at)).long()
        live = ok.any(1)
        logp = torch.gather(torch.log_softmax(z, 1), 1, at)
        x = s["teacher"].to(_D) * c["scale"]
        if s["teacher_lse"] is None:
            norm = torch.logsumexp(torch.where(ok, x, -_INF), 1)
            norm = torch.where(live, norm, torch.zeros_like(norm))
        else:
            norm = s["teacher_lse"].to(_D)
        x = x - norm[:, None]
        nll = torch.where(ok, x.exp() * (x - logp), torch.zeros_like(x)).sum(1)
        w = live.to(_D) if s["weights"] is None else s["weights"].to(_D) * live
        total = (w * nll).sum()
        if c["reduction"] == "mean" and bool(live.any()):
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


def _exact_embed(c, seed):
    s = _embed_inputs(c, seed)
    ids = s["ids"].long()
    if not c["backward"]:
        padded = torch.cat([s["table"].to(_D), torch.zeros(1, c["H"], dtype=_D, device="cuda")])
        return {"out": padded[torch.where(ids < 0, c["V"], ids)] * c["scale"]}
    d = torch.zeros(c["V"] + 1, c["H"], dtype=_D, device="cuda")
    d.index_put_((torch.where(ids < 0, c["V"], ids),), s["d_out"].to(_D), accumulate=True)
    d = d[:-1] * c["scale"]
    return {"d_table": d if s["add"] is None else d + s["add"].to(_D)}


def exact(case, seed):
    return {"sample": _exact_sample, "top": _exact_top, "distill": _exact_distill,
            "embed": _exact_embed}[case["op"]](case, seed)
