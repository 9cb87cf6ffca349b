"""Every output of the training operators is written, whatever the memory held before: NaN
stands in all of them when the call is made."""
import dataclasses

import pytest
import torch

from test_gpu_train import LOSS_CASES, check_loss, run_loss

pytestmark = pytest.mark.gpu


def _again_over_nan(out, args):
    from dspark_block_drafter_gb300 import torch_io as tio
    for f in dataclasses.fields(out):
        t = getattr(out, f.name)
        if t is not None:
            t.fill_(float("nan") if t.is_floating_point() else -77)
    tio.head_loss(*args)
    assert tio.device_status(args[6]) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
@pytest.mark.parametrize("pieces", [1, 2])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 20, 128, 129, 600])
def test_gradients_of_no_rows_are_zero(T, reduction, pieces, form, dtype):
    out, _, args = run_loss(T, 72, 1504, 8, dtype, form=form, n_emit=600, ignored=T,
                            pieces=pieces, reduction=reduction)
    _again_over_nan(out, args)
    assert int(out.n_rows) == 0
    for name in ("loss", "total", "d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2"):
        t = getattr(out, name)
        assert bool((t == 0).all()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LOSS_CASES + [
    dict(T=T, H=72, V=1504, r=8, ignored=T // 2, grads=grads) for T in (1, 8, 9, 16)
    for grads in ("all", "frozen")], ids=str)
def test_loss_writes_every_output(case, dtype):
    out, o, args = run_loss(dtype=dtype, seed=3, **case)
    _again_over_nan(out, args)
    check_loss(out, o, dtype)
