"""Gate rows shared by many rows: spans up to the largest int, and those of large batches,
where a CTA sums a whole span, several parts of one, or several rows at a time."""
import pytest
import torch

from test_gpu_train import run_norm

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 16, 1100])
def test_one_gate_row_for_every_row(T, dtype):
    """A span longer than the batch is one of the batch's length."""
    from dspark_block_drafter_gb300 import torch_io as tio
    tio_, cfg, x, y, w_pre, h, xo, kw = run_norm(T, 136, dtype, span=MOST)
    grads = []
    for span in (T, T + 1, 2 ** 30, MOST - T, MOST - 1, MOST):
        c = tio.make_norm_config(T, 136, dtype, 1e-6, 0.5, 1.0, span)
        out = tio.NormGrads.allocate(c)
        ws = tio.norm_workspace_for(c)
        tio.block_norm_backward(c, x, y, w_pre, h, out, ws, d_x_out=xo, **kw)
        grads.append(out)
    for g in grads[1:]:
        for name in ("d_x", "d_y", "d_gate", "d_w_post", "d_w_pre"):
            assert torch.equal(getattr(g, name), getattr(grads[0], name)), name
