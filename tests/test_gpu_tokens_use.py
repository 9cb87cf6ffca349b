"""The operators on tokens and the distillation as programs use them: in graphs, on streams, twice,
into parts of larger arrays, past 2^31 elements, and one after the other."""
import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(g, T, V, dtype=torch.float32):
    z = -1.2 * (torch.rand(T, V, generator=g, device="cuda") * V + 1).log() + 15
    return (z + 0.5 * torch.randn(T, V, generator=g, device="cuda")).to(dtype)


def _distill_state(g, T=96, H=128, V=2000, r=16, k=12, dtype="bf16"):
    from dspark_block_drafter_gb300 import torch_io as tio
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    head = tio.Head(randn(V, H, std=0.1), randn(V, r, std=0.3), randn(r, V, std=0.3))
    cfg = tio.make_loss_config(T, H, V, r, dtype)
    out = tio.LossOutputs.allocate(cfg, head)
    z = _logits(g, T, V)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    values, lse = torch.empty(T, k, device="cuda"), torch.empty(T, device="cuda")
    teacher = tio.Teacher(ids, values, lse)
    prev = torch.randint(V, (T,), generator=g, device="cuda").int()
    return dict(cfg=cfg, head=head, out=out, z=z, teacher=teacher, prev=prev,
                hidden=randn(T, H), ws=tio.distill_workspace_for(cfg, head, teacher, out))


def _calls():
    """name -> (inputs that are refilled, outputs, the call with a stream)."""
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(1)
    calls = {}
    for name, T, V in (("sample_held", 7, 9000), ("sample_one_cta", 70, 70000)):
        z, u = _logits(g, T, V), torch.rand(T, generator=g, device="cuda")
        tok, lp = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
        cfg = tio.make_sample_config(T, V, "f32", top_k=40, top_p=0.9)
        calls[name] = ([z, u], [tok, lp], lambda s=None, a=(cfg, z, u, tok), lp=lp:
                       tio.sample(*a, logp=lp, stream=s))
    for name, T, V in (("top_held", 5, 30000), ("top_one_cta", 66, 60000)):
        z = _logits(g, T, V, torch.bfloat16)
        ids, val = torch.empty(T, 9, dtype=torch.int32, device="cuda"), torch.empty(T, 9, device="cuda")
        lse = torch.empty(T, device="cuda")
        calls[name] = ([z], [ids, val, lse], lambda s=None, a=(z, ids, val), lse=lse:
                       tio.top_logits(*a, lse=lse, stream=s))
    table = torch.randn(300, 64, generator=g, device="cuda")
    ids = torch.randint(300, (50,), generator=g, device="cuda").int()
    out = torch.empty(50, 64, device="cuda")
    ecfg = tio.make_embed_config(50, 300, 64, "f32", scale=2.0)
    calls["embed"] = ([table], [out], lambda s=None: tio.embed(ecfg, table, ids, out, stream=s))
    for name, T in (("embed_backward", 5000), ("embed_backward_many", 20000)):
        ids_b = torch.randint(300, (T,), generator=g, device="cuda").int()
        d = torch.randn(T, 64, generator=g, device="cuda")
        base, grad = torch.randn(300, 64, generator=g, device="cuda"), torch.empty(300, 64, device="cuda")
        bcfg = tio.make_embed_config(T, 300, 64, "f32")
        ws = tio.embed_workspace_for(bcfg)
        calls[name] = ([d, base], [grad], lambda s=None, a=(bcfg, ids_b, d, grad, ws), base=base:
                       tio.embed_backward(*a, add=base, stream=s))
    for dtype in ("f32", "bf16"):
        s = _distill_state(g, dtype=dtype)
        o = s["out"]
        tio.top_logits(s["z"], s["teacher"].ids, s["teacher"].logits, lse=s["teacher"].lse)
        calls["distill_" + dtype] = (
            [s["hidden"], s["teacher"].logits],
            [o.loss, o.total, o.d_hidden, o.d_lm_head, o.d_markov_w1, o.d_markov_w2],
            lambda st=None, s=s: tio.distill_loss(s["cfg"], s["head"], s["teacher"], s["hidden"],
                                                  s["prev"], s["out"], s["ws"], stream=st))
    return calls


NAMES = ["sample_held", "sample_one_cta", "top_held", "top_one_cta", "embed", "embed_backward",
         "embed_backward_many", "distill_f32", "distill_bf16"]


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """A graph reads its inputs anew, and gives the bits of a direct call; the same call twice
    too, and one on another stream."""
    ins, outs, call = _calls()[name]
    call()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    for o in outs:
        o.fill_(-3)
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for x in ins:
        x.copy_(x.roll(1, 0))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [o.clone() for o in outs]
    assert not all(torch.equal(a, b) for a, b in zip(first, replayed))
    for o in outs:
        o.fill_(-3)
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, outs))
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, outs))


def test_two_graphs_share_a_workspace():
    """Two captured calls of different sizes, replayed in turn on one stream."""
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(2)
    cases = []
    for T, V, H in ((5000, 700, 40), (300, 2000, 24)):
        ids = torch.randint(V, (T,), generator=g, device="cuda").int()
        d, out = torch.randn(T, H, generator=g, device="cuda"), torch.empty(V, H, device="cuda")
        cases.append((tio.make_embed_config(T, V, H, "f32"), ids, d, out))
    ws = max((tio.embed_workspace_for(c[0]) for c in cases), key=lambda w: w.numel())
    want = []
    for c in cases:
        tio.embed_backward(*c, ws)
        torch.cuda.synchronize()
        want.append(c[3].clone())
    graphs = []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tio.embed_backward(*c, ws)
    for i in (0, 1, 1, 0, 0, 1):
        cases[i][3].fill_(7)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(cases[i][3], want[i])


def test_overlapping_calls_on_two_streams():
    """Sampling and top logits keep nothing between calls: many at once give each its own."""
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(3)
    T, V = 24, 50000
    streams = [torch.cuda.Stream() for _ in range(3)]
    zs = [_logits(g, T, V) for _ in range(12)]
    u = torch.rand(T, generator=g, device="cuda")
    cfg = tio.make_sample_config(T, V, "f32", top_p=0.95)
    alone, both = [], []
    for z in zs:
        alone.append(torch.empty(T, dtype=torch.int32, device="cuda"))
        tio.sample(cfg, z, u, alone[-1])
    torch.cuda.synchronize()
    both = [torch.empty_like(a) for a in alone]
    for i, z in enumerate(zs):
        tio.sample(cfg, z, u, both[i], stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, both))


def test_nothing_is_written_beside_the_outputs():
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(4)
    for T, V in ((9, 5000), (80, 50000)):
        z, u = _logits(g, T, V), torch.rand(T, generator=g, device="cuda")
        tok = torch.full((T + 2,), -9, dtype=torch.int32, device="cuda")
        lp = torch.full((T + 2,), -9.0, device="cuda")
        tio.sample(tio.make_sample_config(T, V, "f32"), z, u, tok[1:-1], logp=lp[1:-1])
        ids = torch.full((T + 2, 7), -9, dtype=torch.int32, device="cuda")
        val, lse = torch.full((T + 2, 7), -9.0, device="cuda"), torch.full((T + 2,), -9.0, device="cuda")
        tio.top_logits(z, ids[1:-1], val[1:-1], lse=lse[1:-1])
        for t in (tok, lp, ids, val, lse):
            assert bool((t[0] == -9).all()) and bool((t[-1] == -9).all())
            assert not bool((t[1:-1] == -9).any())
    for dtype in (torch.float32, torch.bfloat16):
        for H in (24, 33):
            full = torch.full((52, H), -9.0, dtype=dtype, device="cuda")
            ids = torch.randint(50, (300,), generator=g, device="cuda").int()
            d = torch.randn(300, H, generator=g, device="cuda").to(dtype)
            cfg = tio.make_embed_config(300, 50, H, "f32" if dtype == torch.float32 else "bf16")
            tio.embed_backward(cfg, ids, d, full[1:-1], tio.embed_workspace_for(cfg))
            assert bool((full[0] == -9).all()) and bool((full[-1] == -9).all())
            out = torch.full((302, H), -9.0, dtype=dtype, device="cuda")
            tio.embed(cfg, full[1:-1], ids, out[1:-1])
            assert bool((out[0] == -9).all()) and bool((out[-1] == -9).all())


def test_rows_of_more_than_2_31_logits():
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V, n = 14400, 151936, 3
    assert T * V > 2 ** 31
    z = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    g = _gen(5)
    for a in range(0, T, 1200):
        z[a:a + 1200] = _logits(g, 1200, V)
    u = torch.rand(T, generator=g, device="cuda")
    tok, lp = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    tio.sample(tio.make_sample_config(T, V, "bf16", top_k=20, top_p=0.9), z, u, tok, logp=lp)
    ids, val = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    tio.top_logits(z, ids, val)
    top = z[-n:].double().cpu().numpy()
    for i in range(n):
        want, logp, near = to.sample_row(top[i], float(u[T - n + i]), top_k=20,
                                         top_p=float(np.float32(0.9)))
        assert near < 2.0 ** -26 or int(tok[T - n + i]) == want
        assert np.array_equal(ids[T - n + i].cpu().numpy(), to.top_row(top[i], 4)[0])
    # all rows: the drawn token is one of the 20 largest, the listed ones the largest
    assert bool((z.gather(1, ids[:, :1].long())[:, 0] == z.max(1).values).all())
    assert bool((tok >= 0).all()) and bool((lp <= 0).all())


def test_tables_of_more_than_2_31_elements():
    from dspark_block_drafter_gb300 import torch_io as tio
    V, H, T = 540000, 4096, 3000
    assert V * H > 2 ** 31
    g = _gen(6)
    ids = torch.randint(V - 500, V, (T,), generator=g, device="cuda").int()
    ids[:7] = torch.tensor([0, 1, V - 1, V - 1, 5, 0, 262143], dtype=torch.int32)
    d = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    grad = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    cfg = tio.make_embed_config(T, V, H, "bf16")
    tio.embed_backward(cfg, ids, d, grad, tio.embed_workspace_for(cfg))
    want = torch.zeros(1000, H, dtype=torch.float64, device="cuda")
    on = ids >= V - 1000
    want.index_add_(0, ids[on].long() - (V - 1000), d[on].double())
    mag = torch.zeros_like(want).index_add_(0, ids[on].long() - (V - 1000), d[on].double().abs())
    off = (grad[-1000:].double() - want).abs()
    assert bool((off <= BF16 * want.abs() + 36 * 2.0 ** -24 * mag * (1 + BF16)).all())
    assert bool((grad[2:5] == 0).all()) and bool((grad[6:262143] == 0).all())
    assert bool((grad[262144:V - 1000] == 0).all())
    assert torch.equal(grad[262143], d[6])
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    tio.embed(cfg, grad, ids, out)
    assert torch.equal(out, grad[ids.long()])


def test_sampled_targets_verify_drafts():
    """The target's logits are sampled, and verify takes the tokens: a draft holds exactly as far as
    it is what was drawn."""
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(7)
    B, N, V = 32, 6, 4000
    z = _logits(g, B * (N + 1), V)
    u = torch.rand(B * (N + 1), generator=g, device="cuda")
    target = torch.empty(B * (N + 1), dtype=torch.int32, device="cuda")
    tio.sample(tio.make_sample_config(B * (N + 1), V, "f32", temperature=0.8, top_k=50, top_p=0.9), z, u,
               target)
    target = target.view(B, N + 1)
    draft = target[:, :N].clone()
    wrong = torch.arange(B, device="cuda") % (N + 1)
    rows = torch.nonzero(wrong < N).flatten()
    draft[rows, wrong[rows]] = (draft[rows, wrong[rows]] + 1) % V
    acc, bonus = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    emitted = torch.empty(B, N + 1, dtype=torch.int32, device="cuda")
    tio.verify(draft.contiguous(), torch.full((B,), N, dtype=torch.int32, device="cuda"), target, acc,
               bonus, emitted)
    assert torch.equal(acc.long(), wrong)
    assert torch.equal(bonus, target[torch.arange(B, device="cuda"), wrong])
    for b in range(B):
        n = int(acc[b]) + 1
        assert torch.equal(emitted[b, :n], target[b, :n]) and bool((emitted[b, n:] == -1).all())


def test_draws_follow_their_probabilities():
    """A grid of uniform numbers draws every kept token as often as its probability says, within
    one draw a border."""
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V = 20000, 50
    z = torch.randn(1, V, generator=_gen(8), device="cuda").expand(T, V).contiguous()
    u = ((torch.arange(T, device="cuda") + 0.5) / T).float()
    tok = torch.empty(T, dtype=torch.int32, device="cuda")
    tio.sample(tio.make_sample_config(T, V, "f32", top_k=30), z, u, tok)
    w = np.exp(z[0].double().cpu().numpy())
    keep = to.order(z[0].cpu().numpy())[:30]
    p = np.zeros(V)
    p[keep] = w[keep] / w[keep].sum()
    seen = np.bincount(tok.cpu().numpy(), minlength=V)
    assert np.all(np.abs(seen - p * T) <= 1.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_training_step_of_a_tied_head(dtype):
    """Embedding, norm, teacher's list, distillation, and the gradients back onto the table that is
    both ends, against the chain in fp64."""
    from dspark_block_drafter_gb300 import torch_io as tio
    g = _gen(9)
    T, H, V, k = 60, 64, 504, 10
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    table = (torch.randn(V, H, generator=g, device="cuda") * 0.3).to(dt)
    w_pre = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dt)
    ids = torch.randint(V, (T,), generator=g, device="cuda").int()
    zt = _logits(g, T, V)
    ecfg, ncfg = tio.make_embed_config(T, V, H, dtype, scale=4.0), tio.make_norm_config(T, H, dtype)
    lcfg = tio.make_loss_config(T, H, V, 0, dtype)
    x, h = torch.empty(T, H, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda")
    head = tio.Head(table, None, None)
    out = tio.LossOutputs.allocate(lcfg, head)
    lids, lval = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    teacher = tio.Teacher(lids, lval)
    ng = tio.NormGrads.allocate(ncfg, gate=False, w_post=False, y=False)
    tio.top_logits(zt, lids, lval)
    tio.embed(ecfg, table, ids, x)
    tio.block_norm(ncfg, x, None, w_pre, h)
    ws = tio.distill_workspace_for(lcfg, head, teacher, out)
    tio.distill_loss(lcfg, head, teacher, h, None, out, ws)
    tio.block_norm_backward(ncfg, x, None, w_pre, out.d_hidden, ng, tio.norm_workspace_for(ncfg))
    head_grad = out.d_lm_head.clone()
    tio.embed_backward(ecfg, ids, ng.d_x, out.d_lm_head, tio.embed_workspace_for(ecfg),
                       add=out.d_lm_head)
    grads = tio.GradList([out.d_lm_head, ng.d_w_pre])
    norm = torch.empty(1, device="cuda")
    tio.clip_grads(grads, 1e6, norm, tio.clip_workspace_for(grads))
    assert tio.device_status(ws) == 0

    D = torch.float64
    t64, w64 = table.to(D).requires_grad_(), w_pre.to(D).requires_grad_()
    e = 4.0 * t64[ids.long()]
    hh = e / (e.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w64
    logp = torch.log_softmax(hh @ t64.t(), 1)
    lq = torch.log_softmax(lval.to(D), 1)
    total = (lq.exp() * (lq - logp.gather(1, lids.long()))).sum(1).mean()
    total.backward()
    # bf16 rounds x, h, d_hidden and d_x (2^-9 each of the whole, and the gradients' products):
    # a few parts in a hundred of the largest entry; fp32 a few times 2^-20
    tol = 2.0 ** -4 if dtype == "bf16" else 2.0 ** -16
    assert abs(float(out.total) - total.item()) <= tol * abs(total.item())
    for got, want in ((out.d_lm_head, t64.grad), (ng.d_w_pre, w64.grad)):
        assert (got.to(D) - want).abs().max().item() <= tol * want.abs().max().item()
        assert (got.to(D) - want).norm() <= tol / 2 * want.norm()
    off = torch.ones(V, dtype=torch.bool, device="cuda")
    off[ids.long()] = False
    assert torch.equal(out.d_lm_head[off], head_grad[off])
    want = (out.d_lm_head.to(D).square().sum() + ng.d_w_pre.to(D).square().sum()).sqrt().item()
    assert abs(float(norm) - want) <= 2.0 ** -18 * want
