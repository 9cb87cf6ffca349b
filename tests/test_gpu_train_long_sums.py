"""Gradients that are sums of very many terms of one sign.

The tensor core cuts its partial sums toward zero: each step of 16 terms loses a unit in the last
place or so of the partial sum, near 1e-7 of the final one.  A sum over 2^20 rows or columns in one
accumulator is short by 0.6%.  The bounds allow the loss 2^-24 a step over 2^16 rows and over 2^18
columns.  The other errors have no sign and average out over the many elements of a gradient: the
output's rounding, 2^-9 / sqrt(3) of an element (uniform within half a unit), and those of the
gradient of the logits, as large and averaged over the terms too: five standard deviations of
both."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROUNDING = 2.0 ** -9 / 3 ** 0.5


def _make(T, H, V, dtype, gen, hidden_std, head):
    from dspark_block_drafter_gb300 import torch_io as tio
    hidden = (torch.randn(T, H, generator=gen, device="cuda").abs() * hidden_std).to(dtype)
    cfg = tio.make_loss_config(T, H, V, 0, "bf16" if dtype is torch.bfloat16 else "f32",
                               reduction="sum", vocab_pieces=1)
    return tio, hidden, cfg, tio.Head(head, None, None)


def _rows_off(T, dtype):
    """Relative errors of d_lm_head's rows that no label names: sums of positive terms."""
    H, V, labelled = 64, 256, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    head = (torch.randn(V, H, generator=g, device="cuda") * 0.02).to(dtype)
    tio, hidden, cfg, head = _make(T, H, V, dtype, g, 1.0, head)
    labels = torch.randint(labelled, (T,), generator=g, device="cuda").int()
    out = tio.LossOutputs.allocate(cfg, head, d_hidden=False)
    ws = tio.loss_workspace_for(cfg, head, out)
    tio.head_loss(cfg, head, hidden, None, labels, out, ws)
    assert tio.device_status(ws) == 0
    want = torch.zeros(V - labelled, H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 16):
        x = hidden[a:a + (1 << 16)].double()
        q = torch.softmax(x @ head.lm_head.double().t(), 1)
        want += q[:, labelled:].t() @ x
    return (out.d_lm_head[labelled:].double() - want) / want


@pytest.mark.parametrize("T", [4000, 70000, 2 ** 20 - 3])
def test_head_gradient_over_many_rows(T):
    off = _rows_off(T, torch.bfloat16)
    lost = min(T, 1 << 16) / 16 * 2.0 ** -24
    assert abs(off.mean().item()) < lost + 5 * ROUNDING * (2 / off.numel()) ** 0.5


def test_hidden_gradient_over_many_columns():
    T, H, V = 4096, 2048, 2 ** 20
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 1 << 16):
        w[a:a + (1 << 16)] = torch.randn(1 << 16, H, generator=g, device="cuda").abs() * 0.02
    w[:4] = 0                                   # the labels' rows: nothing is taken off the sum
    tio, hidden, cfg, head = _make(T, H, V, torch.bfloat16, g, 1.0, w)
    labels = torch.randint(4, (T,), generator=g, device="cuda").int()
    out = tio.LossOutputs.allocate(cfg, head)     # (with d_lm_head: one split of the columns)
    ws = tio.loss_workspace_for(cfg, head, out)
    tio.head_loss(cfg, head, hidden, None, labels, out, ws)
    assert tio.device_status(ws) == 0
    x = hidden[:8].double()
    z = torch.cat([x @ w[a:a + (1 << 16)].double().t() for a in range(0, V, 1 << 16)], 1)
    q = torch.softmax(z, 1)
    want = sum(q[:, a:a + (1 << 16)] @ w[a:a + (1 << 16)].double() for a in range(0, V, 1 << 16))
    off = (out.d_hidden[:8].double() - want) / want
    lost = 2 ** 18 / 16 * 2.0 ** -24
    assert abs(off.mean().item()) < lost + 5 * ROUNDING * (2 / off.numel()) ** 0.5


# fp32: chains of up to 4096 additions, then one of the parts.  An addition rounds to nearest, 2^-24
# of its partial sum at most: 2^-24 / sqrt(3) rms, of a partial sum that is 1 / sqrt(3) of the last
# (rms); six deviations, and 2^-21 for the gradient of the logits.
def _chain_bound(n):
    parts = max(1.0, n / 4096)
    return 6 * 2.0 ** -24 / 3 * (min(n, 4096) / parts + parts) ** 0.5 + 2.0 ** -21


@pytest.mark.parametrize("T", [4000, 70000, 2 ** 20 - 3])
def test_head_gradient_over_many_rows_f32(T):
    assert _rows_off(T, torch.float32).abs().max().item() < _chain_bound(T)


# (few rows and features: the columns are split among many CTAs; many: hardly; up to 16 rows take
# other kernels)
@pytest.mark.parametrize("T,H,V", [(300, 64, 4000), (300, 64, 2 ** 20 + 5), (4100, 256, 2 ** 20 + 5),
                                   (16, 16384, 2 ** 19 + 3)])
def test_hidden_gradient_over_many_columns_f32(T, H, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    w = torch.empty(V, H, device="cuda")
    for a in range(0, V, 1 << 16):
        b = min(V, a + (1 << 16))
        w[a:b] = torch.randn(b - a, H, generator=g, device="cuda").abs() * 0.16 / H ** 0.5
    w[:4] = 0                                   # the labels' rows: nothing is taken off the sum
    tio, hidden, cfg, head = _make(T, H, V, torch.float32, g, 1.0, w)
    out = tio.LossOutputs.allocate(cfg, head, d_lm_head=False)
    ws = tio.loss_workspace_for(cfg, head, out)
    labels = torch.randint(4, (T,), generator=g, device="cuda").int()
    tio.head_loss(cfg, head, hidden, None, labels, out, ws)
    assert tio.device_status(ws) == 0
    x = hidden[-64:].double()
    z = torch.cat([x @ c.double().t() for c in w.split(1 << 16)], 1)
    q = torch.softmax(z, 1).split(1 << 16, 1)
    want = sum(a @ c.double() for a, c in zip(q, w.split(1 << 16)))
    assert ((out.d_hidden[-64:].double() - want) / want).abs().max().item() < _chain_bound(V)


@pytest.mark.parametrize("T", [4000, 2 ** 20 - 3])
def test_markov_gradient_of_one_prev_over_many_rows_f32(T):
    """markov_w1's row of the token before every slot: eight chains of rows, joined."""
    from dspark_block_drafter_gb300 import torch_io as tio
    H, V, r = 16, 64, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    hidden = torch.randn(T, H, generator=g, device="cuda")
    w, w1 = (torch.randn(V, n, generator=g, device="cuda") * 0.1 for n in (H, r))
    w2 = torch.rand(r, V, generator=g, device="cuda") + 0.1
    w2[:, :4] = 0                               # the labels' columns: nothing is taken off the sum
    labels = torch.randint(4, (T,), generator=g, device="cuda").int()
    prev = torch.full((T,), 7, device="cuda", dtype=torch.int32)
    head = tio.Head(w, w1, w2)
    cfg = tio.make_loss_config(T, H, V, r, "f32", reduction="sum")
    out = tio.LossOutputs.allocate(cfg, head, d_hidden=False, d_lm_head=False)
    ws = tio.loss_workspace_for(cfg, head, out)
    tio.head_loss(cfg, head, hidden, prev, labels, out, ws)
    assert tio.device_status(ws) == 0
    z = hidden.double() @ w.double().t() + (w1[7].double() @ w2.double())[None]
    want = (torch.softmax(z, 1) @ w2.double().t()).sum(0)
    assert ((out.d_markov_w1[7].double() - want) / want).abs().max().item() < _chain_bound(T / 8)


@pytest.mark.parametrize("T", [4000, 2 ** 20 - 3])
def test_gate_gradient_over_many_rows_f32(T):
    """One gate row for every row, and no gradient of h: d_gate = s sum d_x_out y."""
    from dspark_block_drafter_gb300 import torch_io as tio
    H = 64
    g = torch.Generator(device="cuda")
    g.manual_seed(15)
    x, y, up = (torch.rand(T, H, generator=g, device="cuda") + 0.1 for _ in range(3))
    gate, w = torch.ones(1, H, device="cuda"), torch.ones(H, device="cuda")
    cfg = tio.make_norm_config(T, H, "f32", gate_span=T)
    out = tio.NormGrads.allocate(cfg, w_post=False)
    tio.block_norm_backward(cfg, x, y, w, torch.zeros_like(x), out, tio.norm_workspace_for(cfg),
                            d_x_out=up, gate=gate)
    want = (up.double() * y.double()).sum(0)
    # chains of 16 rows, of 256 of those, and of the rest
    rest = max(1.0, T / 4096)
    bound = 6 * 2.0 ** -24 / 3 * (16 + 256 + rest) ** 0.5 + 2.0 ** -23
    assert ((out.d_gate[0].double() - want) / want).abs().max().item() < bound
