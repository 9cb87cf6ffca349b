"""The training operators where offsets pass 32 bits: more than 2^31 elements in the kept
values of the loss, in a norm's rows and in one gradient.  References are computed on the
GPU with torch in fp64, for the rows furthest from the start; bounds as in
test_gpu_train.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def _near(got, want, bound):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), (off - bound).max().item()


def test_loss_of_more_than_2_31_logits():
    from dspark_block_drafter_gb300 import torch_io as tio
    T, H, V = 16500, 64, 151936
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def randn(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    hidden, W = randn(T, H, std=1.0), randn(V, H, std=0.2)
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    head = tio.Head(W, None, None)
    cfg = tio.make_loss_config(T, H, V, 0, "bf16", reduction="sum", vocab_pieces=1)
    out = tio.LossOutputs.allocate(cfg, head)
    ws = tio.loss_workspace_for(cfg, head, out)
    assert T * V > 2 ** 31 and ws.numel() > 2 * T * V
    tio.head_loss(cfg, head, hidden, None, labels.int(), out, ws)
    assert tio.device_status(ws) == 0

    x, w = hidden.double(), W.double()
    lse = torch.cat([torch.logsumexp(x[a:a + 1024] @ w.t(), 1) for a in range(0, T, 1024)])
    want = lse - (x * w[labels]).sum(1)
    dz = 2.0 ** -21 * (x.abs().sum(1).max() * w.abs().max()) + 2.0 ** -20
    _near(out.loss, want, 2 * dz + 2.0 ** -22 * want.abs())
    eps = BF16 + 2.0 ** -11 + 2 * dz + 2.0 ** -20
    # the last rows of d_hidden
    n = 96
    q = torch.exp(x[-n:] @ w.t() - lse[-n:, None])
    q[torch.arange(n), labels[-n:]] -= 1
    ref = q @ w
    _near(out.d_hidden[-n:], ref, BF16 * ref.abs() + eps * (q.abs() @ w.abs()) * (1 + BF16))
    # the last rows of d_lm_head
    q = torch.exp(x @ w[-n:].t() - lse[:, None])
    q -= (labels[:, None] == torch.arange(V - n, V, device="cuda")[None]).double()
    ref = q.t() @ x
    _near(out.d_lm_head[-n:], ref, BF16 * ref.abs() + eps * (q.abs().t() @ x.abs()) * (1 + BF16))


def test_norm_of_more_than_2_31_elements():
    from dspark_block_drafter_gb300 import torch_io as tio
    T, H, n = 530000, 4096, 64
    assert T * H > 2 ** 31
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x[-n:] = torch.randn(n, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    cfg = tio.make_norm_config(T, H, "bf16")
    h = torch.empty_like(x)
    tio.block_norm(cfg, x, x, w, h, w_post=w)
    a, wd = x[-n:].double(), w.double()

    def rms(t):
        return t / (t.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * wd

    ref = rms(a + rms(a))
    _near(h[-n:], ref, BF16 * ref.abs() + 2.0 ** -16 * wd.abs())
    assert not h[:1000].any()
    out = tio.NormGrads.allocate(cfg, gate=False)
    tio.block_norm_backward(cfg, x, x, w, x, out, tio.norm_workspace_for(cfg), w_post=w)
    with torch.enable_grad():
        p, y = a.clone().requires_grad_(), a.clone().requires_grad_()
        u = y / (y.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * wd
        z = p + u
        (z / (z.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * wd * a).sum().backward()
    for got, want in ((out.d_x[-n:], p.grad), (out.d_y[-n:], y.grad)):
        scale = want.pow(2).mean(1, keepdim=True).sqrt()
        _near(got, want, BF16 * want.abs() + 2.0 ** -12 * scale)
    assert not out.d_x[:1000].any()


def test_clip_of_more_than_2_31_elements():
    from dspark_block_drafter_gb300 import torch_io as tio
    n = 2 ** 31 + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[0], t[-1], t[2 ** 31 + 5] = 3.0, 4.0, 12.0
    gl = tio.GradList([t])
    norm = torch.empty(1, device="cuda")
    tio.clip_grads(gl, 6.5, norm, tio.clip_workspace_for(gl))
    assert abs(float(norm) - 13.0) < 1e-5
    assert (float(t[0]), float(t[-1]), float(t[2 ** 31 + 5])) == (1.5, 2.0, 6.0)
    assert int(t.count_nonzero()) == 3
