"""Distillation of the same inputs gives the same bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _tensor(rng, *shape, std=1.0, dtype="f32"):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).cuda().to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["full", "d2t"])
def test_distill_repeats_its_bits(form, dtype):
    """Again, and with a call on other tensors in between, waiting for nothing."""
    from dspark_block_drafter_gb300 import torch_io as tio

    def make(seed):
        rng = np.random.default_rng(seed)
        T, H, V, r, k = 333, 128, 6016, 40, 17
        emit = np.sort(rng.permutation(V)[:4008]).astype(np.int32)
        rows = len(emit) if form == "d2t" else V
        head = tio.Head(_tensor(rng, rows, H, std=0.1, dtype=dtype),
                        _tensor(rng, V, r, std=0.3, dtype=dtype),
                        _tensor(rng, r, rows, std=0.3, dtype=dtype), None,
                        torch.from_numpy(emit).cuda() if form == "d2t" else None)
        ids = np.stack([rng.permutation(V)[:k] for _ in range(T)]).astype(np.int32)
        ids[rng.uniform(size=T) < 0.3] = -1
        teacher = tio.Teacher(torch.from_numpy(ids).cuda(), _tensor(rng, T, k, std=3.0))
        cfg = tio.make_loss_config(T, H, V, r, dtype, "sum", vocab_pieces=4)
        out = tio.LossOutputs.allocate(cfg, head)
        ws = tio.distill_workspace_for(cfg, head, teacher, out)
        prev = torch.from_numpy(rng.integers(0, 40, T).astype(np.int32)).cuda()
        weights = torch.from_numpy(rng.uniform(0.5, 1.5, T).astype(np.float32)).cuda()
        return (cfg, head, teacher, _tensor(rng, T, H, dtype=dtype), prev, out, ws, weights)

    mine, other = make(1), make(2)
    names = ("loss", "total", "d_hidden", "d_lm_head", "d_markov_w1", "d_markov_w2")
    tio.distill_loss(*mine)
    torch.cuda.synchronize()
    first = [getattr(mine[5], n).clone() for n in names]
    for _ in range(5):
        tio.distill_loss(*mine)
        tio.distill_loss(*other)
        tio.distill_loss(*mine)
        torch.cuda.synchronize()
        for n, t in zip(names, first):
            assert torch.equal(getattr(mine[5], n), t), n
