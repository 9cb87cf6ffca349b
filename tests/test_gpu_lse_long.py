"""Log-sum-exps of rows of any length."""
import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lse(z, dtype="f32", T=1, k=8):
    from dspark_block_drafter_gb300 import torch_io as tio
    x = torch.from_numpy(z.astype(np.float32)).cuda().to(DT[dtype]).expand(T, -1).contiguous()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    values, sums = torch.empty(T, k, device="cuda"), torch.empty(T, device="cuda")
    tio.top_logits(x, ids, values, lse=sums)
    return x[0].double().cpu().numpy(), sums.double().cpu().numpy()


def _check_lse(z, dtype="f32", T=1, k=8):
    x, got = _lse(z, dtype, T, k)
    want = to.top_row(x, 1)[2]
    on = x > -np.inf
    p = np.exp(x[on] - want)
    away = np.sum(p * np.abs(x[on] - np.max(x[on])))
    # An exponent is rounded three times; the exponential, and the factor that brings a CTA's sum
    # to the row's reference, are off by 2^-22 of themselves.  A thread's sum: 8 elements to one
    # value, chains of 32 of those, and the chains' sums with their rounding errors; then the
    # threads' (5 steps), the warps' (16), the CTAs' (8): 64 roundings whatever the length.  The
    # maximum and the logarithm are added, and scaled.
    bound = 2.0 ** -21 + 3 * 2.0 ** -24 * away + 64 * 2.0 ** -24
    assert np.all(np.abs(got - want) <= bound + 2.0 ** -22 * abs(want) + 2.0 ** -22), got - want


@pytest.mark.parametrize("a", [0.04, 0.13, 0.24, 0.25, 0.56, 0.66])
@pytest.mark.parametrize("V,k", [(8_000_000, 8), (8_000_000, 300), (1 << 24, 8)])
def test_log_sum_exp_of_a_long_row_of_near_equal_logits(V, k, a):
    """Equal sums of vectors, one after the other: their roundings go one way within an octave (a
    plain fp32 sum of 3906 of them is off by up to 5e-5 of itself)."""
    z = np.full(V, -a)
    z[::4] = 0.0
    _check_lse(z, k=k)
    z[1] = np.nan
    _check_lse(z, k=k)


@pytest.mark.parametrize("step", [1e-9, 1e-7, 1e-5, -1e-7])
def test_log_sum_exp_of_a_long_row_that_rises(step):
    """Nearly every vector has a new maximum."""
    V = 8_000_000
    _check_lse(np.arange(V) * step)
    _check_lse(np.arange(V) * step * 100 - 3.0, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_log_sum_exp_of_rows_in_a_batch(dtype):
    rng = np.random.default_rng(2)
    for T in (3, 70):
        for V in (4099, 151936, 300001):
            _check_lse(rng.normal(size=V) * 3 + 15, dtype, T)
            z = rng.normal(size=V)
            z[V // 3:] = -np.inf
            z[: V // 7] -= 60.0
            z[V - 1] = 40.0
            _check_lse(z, dtype, T)
