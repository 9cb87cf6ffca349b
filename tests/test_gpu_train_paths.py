"""Paths of the training operators that take larger batches than the other tests have: gate rows
whose gradient is stored straight from registers, more rows of one previous token than a warp
looks at in one step, and bias-form heads whose rows are compacted by one CTA."""
import pytest

from test_gpu_train import check_loss, run_loss, run_norm

pytestmark = pytest.mark.gpu


# a CTA takes T / 512 rows of a gate row at a time from 1024 rows on, 16 from 8192: spans up to
# that are one part
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 57, 130])
@pytest.mark.parametrize("T,span", [(1024, 2), (1023, 2), (1600, 3), (1601, 2), (4099, 8), (4099, 7),
                                    (8192, 16), (8200, 16), (8193, 7), (8192, 17), (8192, 33)])
def test_norm_gate_rows_of_one_part(T, span, H, dtype):
    run_norm(T, H, dtype, span=span)


def test_norm_gate_rows_of_one_part_wide():
    run_norm(1100, 2816, "bf16", span=2)
    run_norm(1100, 2816, "bf16", span=2, up=False)
    run_norm(1100, 2816, "bf16", span=2, post=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("prev_range", [1, 7, 1000])
@pytest.mark.parametrize("T,r", [(2100, 40), (1025, 300), (4200, 8)])
def test_loss_many_rows_of_one_prev(T, r, prev_range, dtype):
    out, o, _ = run_loss(T, 64, 1000, r, dtype, prev_range=prev_range, ignored=T // 9,
                         weighted=True)
    check_loss(out, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pieces", [1, 3])
@pytest.mark.parametrize("T,ignored", [(513, 0), (700, 101), (4200, 3000), (5000, 4999)])
def test_loss_bias_form_of_many_rows(T, ignored, pieces, dtype):
    out, o, _ = run_loss(T, 64, 3000, 16, dtype, form="bias", n_emit=1301, ignored=ignored,
                         pieces=pieces, poison=True)
    check_loss(out, o, dtype)
