"""How much workspace the loss asks for: what the header says is held, and no more."""
import os

import pytest

import dspark_block_drafter_gb300 as ds
from dspark_block_drafter_gb300 import _abi


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from dspark_block_drafter_gb300 import build
        build.build()
    return ds.lib()


def _size(T, H, V, r, dtype, pieces, names):
    cfg = _abi.dspark_loss_config(T=T, H=H, V=V, r=r, dtype=dtype, reduction=1,
                                  vocab_pieces=pieces, loss_scale=1.0)
    head = _abi.dspark_head(lm_head=0x10000, V_head=V, markov_w1=0x10000, markov_w2=0x10000)
    out = _abi.dspark_loss_outputs(**{n: 0x10000 for n in names})
    return ds.dspark_head_loss_workspace_size(cfg, head, out)


@pytest.mark.parametrize("dtype", [_abi.DSPARK_F32, _abi.DSPARK_BF16])
@pytest.mark.parametrize("names", [["d_hidden"], ["d_hidden", "d_lm_head", "d_markov_w1",
                                                  "d_markov_w2"]])
@pytest.mark.parametrize("H,r", [(64, 0), (1024, 72), (4096, 256), (8192, 512)])
@pytest.mark.parametrize("T", [1, 129, 4096, 16384, 65536, 1 << 20])
def test_pieces_bound_the_workspace(T, H, r, names, dtype):
    V = 151936
    if r == 0:
        names = [n for n in names if "markov" not in n]
    es = 4 if dtype == _abi.DSPARK_F32 else 2
    rows = (T + 255) // 256 * 256
    x = H + (r + 63) // 64 * 64
    stats = 8 * ((V + (63 if es == 4 else 127)) // (64 if es == 4 else 128))
    piece = (V + 4) // 5 // 256 * 256 + 512
    need = rows * (es * x + stats + 32 + es * piece)      # X, the statistics, rows, one piece
    # fp32 partial sums of X's gradient: once for every row, or 512 MB (fp32 heads: once, or
    # enough 64 x 64 tiles for 608 CTAs)
    need += max(4 * rows * x, 1 << 29) if es == 2 else 4 * rows * x + 608 * 256 * 64 * 4
    assert 0 < _size(T, H, V, r, dtype, 5, names) <= need + (1 << 16)


def test_partial_sums_have_their_room_where_it_is_small():
    """One piece of 512 rows: seven splits of dX are taken, and more may be."""
    with_dx = _size(512, 4096, 151936, 256, 1, 1, ["d_hidden", "d_markov_w1"])
    without = _size(512, 4096, 151936, 256, 1, 1, ["d_lm_head"])
    assert with_dx - without >= 7 * 512 * 4352 * 4
