"""The training operators' C ABI without a GPU: refusals come before any launch."""
import ctypes

import pytest

import dspark_block_drafter_gb300 as ds
from dspark_block_drafter_gb300 import _abi

I, U, W = _abi.DSPARK_ERR_INVALID_ARG, _abi.DSPARK_ERR_UNSUPPORTED, _abi.DSPARK_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(_abi.LIB_PATH):
        from dspark_block_drafter_gb300 import build
        build.build()
    return ds.lib()


def _cfg(**kw):
    c = dict(T=5, H=64, V=1000, r=8, dtype=_abi.DSPARK_F32, reduction=_abi.DSPARK_LOSS_MEAN,
             vocab_pieces=0, loss_scale=1.0)
    c.update(kw)
    return _abi.dspark_loss_config(**c)


def _head(**kw):
    h = dict(lm_head=0x1000, lm_bias=None, d2t=None, V_head=1000, markov_w1=0x2000,
             markov_w2=0x3000)
    h.update(kw)
    return _abi.dspark_head(**h)


def _out(**kw):
    o = dict(loss=0x100, total=0x200)
    o.update(kw)
    return _abi.dspark_loss_outputs(**o)


def _loss(cfg, head, out, hidden=0x4000, prev=0x5000, labels=0x6000, ws=0x10000, n=None):
    if n is None:
        n = ds.dspark_head_loss_workspace_size(cfg, head, out)
    return ds.dspark_head_loss(cfg, head, hidden, prev, labels, None, out, ws, n)


def test_struct_layouts_match_c():
    assert ctypes.sizeof(_abi.dspark_loss_config) == 32
    assert ctypes.sizeof(_abi.dspark_loss_outputs) == 56
    assert ctypes.sizeof(_abi.dspark_norm_config) == 28
    assert ctypes.sizeof(_abi.dspark_grad) == 32


@pytest.mark.parametrize("cfg,head,out,status", [
    (dict(T=0), {}, {}, I), (dict(H=0), {}, {}, I), (dict(V=0), {}, {}, I),
    (dict(r=-1), {}, {}, I), (dict(dtype=7), {}, {}, I), (dict(reduction=2), {}, {}, I),
    (dict(vocab_pieces=-1), {}, {}, I), (dict(loss_scale=float("nan")), {}, {}, I),
    (dict(loss_scale=float("inf")), {}, {}, I),
    ({}, dict(lm_head=None), {}, I), ({}, dict(markov_w1=None), {}, I),
    ({}, dict(markov_w2=None), {}, I), ({}, dict(V_head=999), {}, I),
    ({}, dict(V_head=1001, d2t=0x10), {}, I), ({}, dict(V_head=0, d2t=0x10), {}, I),
    (dict(r=0), {}, dict(d_markov_w1=0x9000), I), (dict(r=0), {}, dict(d_markov_w2=0x9000), I),
    (dict(r=513), {}, {}, U), (dict(T=(1 << 20) + 1), {}, {}, U), (dict(H=(1 << 16) + 8), {}, {}, U),
    (dict(dtype=1, H=60), {}, {}, U),
    (dict(dtype=1), dict(V_head=999, d2t=0x10), {}, U),
    (dict(dtype=1), {}, dict(d_lm_head=0x9008), I), (dict(dtype=1), {}, dict(d_markov_w1=0x9008), I),
    (dict(dtype=1), {}, dict(d_markov_w2=0x9004), I),
    (dict(dtype=1), dict(lm_head=0x1002), {}, I), (dict(dtype=1), dict(markov_w2=0x3008), {}, I),
])
def test_loss_refusals(cfg, head, out, status):
    c, h, o = _cfg(**cfg), _head(**head), _out(**out)
    assert ds.dspark_head_loss_workspace_size(c, h, o) == 0
    assert _loss(c, h, o, n=1 << 40) == status
    assert ds.dspark_last_error()


def test_loss_call_refusals():
    c, h, o = _cfg(), _head(), _out(d_hidden=0x7000)
    need = ds.dspark_head_loss_workspace_size(c, h, o)
    assert need > 0 and need % 256 == 0
    assert _loss(c, h, o, hidden=None) == I
    assert _loss(c, h, o, labels=None) == I
    assert _loss(c, h, o, prev=None) == I
    assert _loss(c, h, _out(loss=None), n=need) == I
    assert _loss(c, h, _out(total=None), n=need) == I
    assert _loss(c, h, o, n=need - 1) == W
    assert _loss(c, h, o, ws=None) == W
    assert _loss(c, h, o, ws=0x10010) == W


def test_loss_workspace_follows_what_is_asked_for():
    def size(out=(), **kw):
        return ds.dspark_head_loss_workspace_size(_cfg(T=512, V=100000, **kw),
                                                  _head(V_head=100000),
                                                  _out(**{k: 0x9000 for k in out}))
    for dtype in (0, 1):
        none, one = size(dtype=dtype), size(["d_hidden"], dtype=dtype)
        pieces = size(["d_hidden"], dtype=dtype, vocab_pieces=4)
        assert none < pieces < one
        # nothing the size of the logits without gradients; a quarter of them in four pieces
        assert none < 512 * 100000 * 2
        assert one - pieces > 0.7 * 512 * 100000 * 2
    # no more pieces than 256-column tiles
    assert size(["d_hidden"], vocab_pieces=391) == size(["d_hidden"], vocab_pieces=10 ** 6)


def _norm(**kw):
    c = dict(T=4, H=64, dtype=0, gate_span=1, eps=1e-6, residual_scale=1.0, weight_offset=0.0)
    c.update(kw)
    return _abi.dspark_norm_config(**c)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), I), (dict(H=0), I), (dict(gate_span=0), I), (dict(dtype=2), I),
    (dict(eps=0.0), I), (dict(eps=float("nan")), I), (dict(eps=float("inf")), I),
    (dict(residual_scale=float("inf")), I), (dict(weight_offset=float("nan")), I),
    (dict(H=8193), U), (dict(T=(1 << 30) + 1), U)])
def test_norm_refusals(kw, status):
    c = _norm(**kw)
    assert ds.dspark_block_norm_workspace_size(c) == 0
    assert ds.dspark_block_norm(c, 1, 1, 1, 1, 1, 1, 1) == status
    assert ds.dspark_block_norm_backward(c, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0x10000,
                                         1 << 40) == status


def test_norm_call_refusals():
    c = _norm()
    need = ds.dspark_block_norm_workspace_size(c)
    p = 0x1000
    assert ds.dspark_block_norm(c, None, p, p, p, p, p, p) == I
    assert ds.dspark_block_norm(c, p, None, p, None, p, p, p) == I      # a gate without y
    assert ds.dspark_block_norm(c, p, None, None, p, p, p, p) == I      # w_post without y
    assert ds.dspark_block_norm(c, p, p, p, p, None, p, p) == I
    assert ds.dspark_block_norm(c, p, p, p, p, p, p, None) == I
    full = [p] * 12                            # x, y, gate, w_post, w_pre, d_h, d_x_out, d_*
    for i, status in ((0, I), (4, I), (5, I), (7, I), (8, I), (9, I), (10, I), (11, I)):
        a = list(full)
        a[i] = None
        assert ds.dspark_block_norm_backward(c, *a, 0x10000, need) == status, i
    assert ds.dspark_block_norm_backward(c, *full, 0x10000, need - 1) == W
    assert ds.dspark_block_norm_backward(c, *full, 0x10010, need) == W
    assert ds.dspark_block_norm_backward(c, *full, None, need) == W


def test_clip_refusals():
    def grads(**kw):
        g = dict(in_=0x1000, out=0x1000, n=10, dtype=0)
        g.update(kw)
        return (_abi.dspark_grad * 1)(_abi.dspark_grad(**g))
    ok = grads()
    need = ds.dspark_clip_grads_workspace_size(1, ok)
    assert need > 0 and need % 256 == 0
    for bad, status in ((dict(n=-1), I), (dict(in_=None), I), (dict(out=None), I),
                        (dict(dtype=5), I), (dict(in_=0x1002), I),
                        (dict(dtype=1, out=0x1001), I), (dict(n=(1 << 38) + 1), U)):
        g = grads(**bad)
        assert ds.dspark_clip_grads_workspace_size(1, g) == 0
        assert ds.dspark_clip_grads(1, g, 1.0, 0x100, 0x10000, need) == status
    assert ds.dspark_clip_grads(0, ok, 1.0, 0x100, 0x10000, need) == I
    assert ds.dspark_clip_grads(1, None, 1.0, 0x100, 0x10000, need) == I
    assert ds.dspark_clip_grads(1, ok, -1.0, 0x100, 0x10000, need) == I
    assert ds.dspark_clip_grads(1, ok, float("nan"), 0x100, 0x10000, need) == I
    assert ds.dspark_clip_grads(1, ok, 1.0, None, 0x10000, need) == I
    assert ds.dspark_clip_grads(1, ok, 1.0, 0x100, 0x10000, need - 1) == W
    assert ds.dspark_clip_grads(1, ok, 1.0, 0x100, 0x10008, need) == W


def test_tensor_checks():
    import torch
    from dspark_block_drafter_gb300 import torch_io as tio
    cfg = tio.make_norm_config(4, 64, "f32")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="w_pre"):
        tio.block_norm(cfg, x, None, torch.zeros(63), x)
    with pytest.raises(ValueError, match="x: "):
        tio.block_norm(cfg, torch.zeros(64, 4).t(), None, torch.zeros(64), x)
    with pytest.raises(ValueError, match="gradient 0"):
        tio.GradList([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError, match="outs"):
        tio.GradList([torch.zeros(3)], [torch.zeros(4)])
