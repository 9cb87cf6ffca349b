"""The training calls refuse arrays that are not aligned to their elements, before any launch
(the kernels would fault on them)."""
import os

import pytest

import dspark_block_drafter_gb300 as ds
from dspark_block_drafter_gb300 import _abi

I = _abi.DSPARK_ERR_INVALID_ARG
P, WS, MOST = 0x10000, 0x20000, 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from dspark_block_drafter_gb300 import build
        build.build()
    return ds.lib()


HEAD = ("lm_head", "lm_bias", "markov_w1", "markov_w2", "d2t")
OUT = ("loss", "total", "n_rows", "d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2")
CALL = ("hidden", "prev", "labels", "weights")
WIDE = ("lm_bias", "d2t", "loss", "total", "n_rows", "prev", "labels", "weights")    # 4 bytes always


def _loss(dtype, name, by):
    def at(n):
        return P + (by if n == name else 0)
    cfg = _abi.dspark_loss_config(T=4, H=64, V=1000, r=8, dtype=dtype, reduction=1, vocab_pieces=0,
                                  loss_scale=1.0)
    head = _abi.dspark_head(V_head=1000, **{n: at(n) for n in HEAD})
    out = _abi.dspark_loss_outputs(**{n: at(n) for n in OUT})
    size = ds.dspark_head_loss_workspace_size(cfg, head, out)
    return size, ds.dspark_head_loss(cfg, head, *[at(n) for n in CALL], out, WS, MOST)


@pytest.mark.parametrize("name", HEAD + OUT + CALL)
@pytest.mark.parametrize("dtype", [_abi.DSPARK_F32, _abi.DSPARK_BF16])
def test_loss_refuses_arrays_across_their_elements(dtype, name):
    size = 4 if dtype == _abi.DSPARK_F32 or name in WIDE else 2
    for by in range(1, size):
        need, status = _loss(dtype, name, by)
        assert status == I and ds.dspark_last_error(), by
        assert need == 0 or name in CALL


NORM = ("x", "y", "gate", "w_post", "w_pre", "x_out", "h")
GRAD = ("x", "y", "gate", "w_post", "w_pre", "d_h", "d_x_out", "d_x", "d_y", "d_gate", "d_w_post",
        "d_w_pre")


@pytest.mark.parametrize("dtype", [_abi.DSPARK_F32, _abi.DSPARK_BF16])
def test_norm_refuses_arrays_across_their_elements(dtype):
    cfg = _abi.dspark_norm_config(T=4, H=64, dtype=dtype, gate_span=1, eps=1e-6,
                                  residual_scale=1.0, weight_offset=0.0)
    size = 4 if dtype == _abi.DSPARK_F32 else 2
    for by in range(1, size):
        for i, name in enumerate(NORM):
            args = [P] * len(NORM)
            args[i] += by
            assert ds.dspark_block_norm(cfg, *args) == I, name
        for i, name in enumerate(GRAD):
            args = [P] * len(GRAD)
            args[i] += by
            assert ds.dspark_block_norm_backward(cfg, *args, WS, MOST) == I, name


def test_clip_refuses_a_norm_across_its_element():
    g = (_abi.dspark_grad * 1)(_abi.dspark_grad(in_=P, out=P, n=10, dtype=0))
    for by in (1, 2, 3):
        assert ds.dspark_clip_grads(1, g, 1.0, P + by, WS, MOST) == I
