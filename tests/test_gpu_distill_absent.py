"""Distillation from lists whose absent entries bring any id."""
import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.double().cpu().numpy()


def _tensor(rng, *shape, std=1.0, dtype="f32"):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).cuda().to(DT[dtype])


@pytest.mark.parametrize("T", [12, 600])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d2t", [False, True])
def test_absent_entries_of_any_id(d2t, dtype, T):
    """A logit of -infinity is absent whatever its id: a list padded from a larger vocabulary."""
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(T)
    H, V, k = 64, 504, 6
    emit = np.sort(rng.permutation(V)[:256]).astype(np.int32) if d2t else np.arange(V, dtype=np.int32)
    W, h = _tensor(rng, len(emit), H, dtype=dtype), _tensor(rng, T, H, std=0.1, dtype=dtype)
    ids = np.stack([rng.permutation(emit)[:k] for _ in range(T)]).astype(np.int32)
    s = rng.normal(size=(T, k)).astype(np.float32)
    none = ids.copy(), s.copy()
    for t, (at, v) in ((2, (3, V)), (4, (0, 2 ** 31 - 1)), (5, (5, V + 100))):
        ids[t, at], s[t, at] = v, -np.inf
        none[0][t, at] = -1
    ids[7], s[7] = V + np.arange(k), -np.inf         # (nothing left: no loss, and no error)
    none[0][7] = -1
    got = []
    for i, x in ((ids, s), none):
        head = tio.Head(W, None, None, None, torch.from_numpy(emit).cuda() if d2t else None)
        cfg = tio.make_loss_config(T, H, V, 0, dtype)
        out = tio.LossOutputs.allocate(cfg, head)
        teacher = tio.Teacher(torch.from_numpy(i).cuda(), torch.from_numpy(x).cuda())
        ws = tio.distill_workspace_for(cfg, head, teacher, out)
        tio.distill_loss(cfg, head, teacher, h, None, out, ws)
        assert tio.device_status(ws) == 0 and int(out.n_rows) == T - 1
        got.append(out)
    for name in ("loss", "total", "d_hidden", "d_lm_head"):
        assert torch.equal(getattr(got[0], name), getattr(got[1], name)), name
    o = to.distill_loss(_np(h), _np(W), ids, s, d2t=emit if d2t else None, V=V)
    assert o["dropped"] == 0 and o["n_rows"] == T - 1
