"""Batches of which few rows carry a loss, and batches whose partial sums of d_hidden have little
room: the splits of the vocabulary follow the rows in use."""
import pytest

from test_gpu_train import check_few_rows, check_loss, run_loss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("grads", ["all", "frozen"])
@pytest.mark.parametrize("case", [
    dict(T=1100, H=256, V=4104, r=40, ignored=800), dict(T=1100, H=256, V=4104, r=40, ignored=1099),
    dict(T=128, H=136, V=9000, r=8, ignored=64), dict(T=128, H=136, V=9000, r=8, ignored=63),
    dict(T=3000, H=512, V=2056, r=16, ignored=2900, form="bias", n_emit=1999, pieces=3),
    dict(T=3000, H=512, V=2056, r=16, ignored=2600, form="d2t", n_emit=2000)], ids=str)
def test_few_of_many_rows(case, grads, dtype):
    out, o, _ = run_loss(dtype=dtype, grads=grads, **case)
    check_loss(out, o, dtype)
    if dtype == "bf16" and case["T"] <= 128 and o["n_rows"] <= 64:
        check_few_rows(out, o)


@pytest.mark.parametrize("ignored", [0, 19000])
def test_rows_beyond_the_room_for_every_split(ignored):
    out, o, _ = run_loss(20000, 2048, 2056, 0, "bf16", ignored=ignored, grads="frozen")
    check_loss(out, o, "bf16")
