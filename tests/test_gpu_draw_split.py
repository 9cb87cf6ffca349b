"""A row's token, however the row is split.

Rows of fewer than 64 are held by clusters, of 64 and more read by one CTA each; an unfiltered
draw of the latter takes its sums in the pass that reads the row, in units of what it has seen of
it.  The weights' units are those of the largest, so the token has to be the same.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _draw(x, u, **settings):
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V = x.shape
    cfg = tio.make_sample_config(T, V, "f32" if x.dtype is torch.float32 else "bf16", **settings)
    tokens = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((T,), 7.0, device="cuda")
    tio.sample(cfg, x, u, tokens, logp=logp)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), logp.double().cpu().numpy()


def _same_token(z, u, dtype, **settings):
    """Of the first rows alone (held by clusters) and of all of them, 64 and 320 (one CTA each, of
    1024 and of 512 threads)."""
    x = torch.from_numpy(z.astype(np.float32)).cuda().to(DT[dtype])
    u = torch.from_numpy(u.astype(np.float32)).cuda()
    n = len(z)
    want, lp = _draw(x, u, **settings)
    assert np.all((want >= 0) & (want < z.shape[1]))
    for T in (64, 320):
        at = torch.arange(T, device="cuda") % n
        tokens, logp = _draw(x[at], u[at], **settings)
        assert np.array_equal(tokens, want[at.cpu().numpy()]), (T, np.sum(tokens[:n] != want))
        # (the other tokens' mass, in a sum that may be off by a unit a weight; log1p of its ratio
        # to the token's, as everywhere)
        assert np.all(np.abs(logp[:n] - lp) <= 2.0 ** -19 * np.abs(lp) + 2.0 ** -26)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("octaves", [1, 3, 9, 26, 40])
def test_draw_of_a_row_with_a_late_maximum(octaves, dtype):
    """The largest logit is the last: what went before was summed in finer units.  Half of the
    numbers draw from the others, whose weights are some 2^17 units (26 octaves down)."""
    rng = np.random.default_rng(octaves)
    n, V = 40, 200003
    z = -octaves * np.log(2.0) + 0.3 * rng.normal(size=(n, V))
    z[:, V - 1] = 0.0
    others = np.exp(z[:, :-1]).sum(1)
    u = rng.uniform(size=n)
    u[::2] *= (others / (others + 1))[::2]
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    _same_token(z, u, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_draw_of_a_row_that_rises(dtype):
    """Every part of the row has a larger logit than the one before, by an octave or so."""
    rng = np.random.default_rng(7)
    n, V = 32, 200003
    z = np.linspace(-1.0, 1.0, V) * rng.uniform(1, 40, (n, 1)) + 0.2 * rng.normal(size=(n, V))
    u = rng.uniform(size=n) ** 8
    _same_token(z, u, dtype)
    _same_token(z[:, ::-1].copy(), u, dtype, temperature=0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_draw_of_a_row_with_a_late_logit_of_any_size(dtype):
    """The last logit leaves the range that the weights of the first ones were made for."""
    n, V = 32, 200003
    z = np.random.default_rng(3).normal(size=(n, V))
    z[:, V - 1] = np.resize([np.inf, 3e38, 1e30, 1e9, 70000.0, 30000.0, 2000.0, 90.0], n)
    _same_token(z, np.random.default_rng(4).uniform(size=n), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("settings", [dict(temperature=0.8), dict(top_p=0.9), dict(top_p=0.999, min_p=0.01),
                                      dict(min_p=0.05), dict(top_k=40, top_p=0.9), dict(top_k=3000)],
                         ids=str)
def test_draw_by_every_filter(settings, dtype):
    rng = np.random.default_rng(len(settings))
    n, V = 40, 150001
    z = -rng.uniform(0.7, 2.2, (n, 1)) * np.log(rng.uniform(size=(n, V)) * V + 1) + 18
    z += rng.normal(size=(n, V)) * 0.5
    _same_token(z, rng.uniform(size=n), dtype, **settings)
