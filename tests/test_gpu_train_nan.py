"""A row whose logits are not numbers shows in everything that it takes part in: its loss, the
total, its own gradient and every gradient of a weight it meets.  The other rows keep theirs."""
import pytest
import torch

from test_gpu_train import run_loss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
@pytest.mark.parametrize("pieces", [1, 3])
@pytest.mark.parametrize("T", [5, 20, 100, 300])
def test_a_row_that_is_not_a_number(T, pieces, form, dtype, bad):
    from dspark_block_drafter_gb300 import torch_io as tio
    out, o, args = run_loss(T, 64, 1504, 8, dtype, form=form, n_emit=1000, pieces=pieces)
    cfg, head, hidden, prev, labels, _, ws, _ = args
    before = [out.loss.clone(), out.d_hidden.clone(), out.d_markov_w1.clone()]
    at = 3
    hidden[at, 7] = bad              # (infinity: the row's logits are infinite, both ways)
    tio.head_loss(*args)
    assert tio.device_status(ws) == 0
    keep = torch.arange(T, device="cuda") != at
    assert torch.isnan(out.total).all() and torch.isnan(out.loss[at])
    assert torch.equal(out.loss[keep], before[0][keep])
    assert torch.isnan(out.d_hidden[at]).all()
    assert torch.equal(out.d_hidden[keep], before[1][keep])
    live = torch.ones(head.V_head, dtype=torch.bool, device="cuda")
    if head.lm_bias is not None:
        live = head.lm_bias > -1e8
    assert torch.isnan(out.d_lm_head[live]).all() and torch.isnan(out.d_markov_w2[:, live]).all()
    assert not out.d_lm_head[~live].any() and not out.d_markov_w2[:, ~live].any()
    follows = torch.zeros(cfg.V, dtype=torch.bool, device="cuda")
    follows[prev[at].long()] = True
    assert torch.isnan(out.d_markov_w1[follows]).all()
    assert torch.equal(out.d_markov_w1[~follows], before[2][~follows])
