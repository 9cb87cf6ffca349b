"""Sampling, top logits and the embedding on a GB300 against their fp64 definitions.

A drawn token is the definition's unless a border lies within 2^-26 of the mass of what it is
compared with: a weight is off by at most 2^-27 of itself, and so are sums of them and their
ratios to 2^-26.  A log-probability is log1p of the ratio of the other tokens' mass to the
token's: 2^-26 from the weights, three fp32 roundings of 2^-24 and log1pf's two steps of 2^-23,
which together stay below 2^-20 of the result.  Besides, a weight is cut to units of 2^-S of the
largest, S = 62 - ceil(log2 V): V weights lose less than V 2^-S of it in all, and as the kept mass
M is no less than the largest weight, the log of the token's share x / M moves by at most
V 2^-S / M (the others' part of M) + 2^-S / x (its own, of no account beside 2^-20 |log x|, since
x is drawn with probability x).  The fp64 definition itself is off by some 2^-50.
"""
import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
NEAR = 2.0 ** -26
INF = float("inf")


def _rows(rng, T, V, kind):
    if kind == "zipf":
        z = -rng.uniform(0.7, 2.2, (T, 1)) * np.log(rng.uniform(size=(T, V)) * V + 1) + 18
        return z + rng.normal(size=(T, V)) * 0.5
    if kind == "flat":
        return rng.normal(size=(T, V)) * 0.3
    if kind == "wide":
        return rng.normal(size=(T, V)) * 40
    if kind == "equal":
        return np.full((T, V), 1.25)
    if kind == "few":               # few different values, many of each
        return rng.integers(0, 4, (T, V)) * 0.5
    assert kind == "low"            # far from zero, where differences round
    return rng.normal(size=(T, V)) * 2 - 1000


def _tensor(z, dtype, pad=0, lead=0):
    """Rows of `pad` more elements, the first at `lead` elements into its memory."""
    T, V = z.shape
    full = torch.full((T, V + pad + lead), 1e9, dtype=DT[dtype], device="cuda")
    part = full[:, lead:lead + V]
    part.copy_(torch.from_numpy(z.astype(np.float32)).cuda())
    return part


def draw(z, u, dtype="f32", pad=0, lead=0, rows=None, **settings):
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V = z.shape
    x = _tensor(z, dtype, pad, lead)
    cfg = tio.make_sample_config(T, V, dtype, **settings)
    tokens = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((T,), 7.0, device="cuda")
    extra = {k: torch.from_numpy(v).cuda() for k, v in (rows or {}).items()}
    tio.sample(cfg, x, torch.from_numpy(u.astype(np.float32)).cuda(), tokens, logp=logp, **extra)
    torch.cuda.synchronize()
    return x.double().cpu().numpy(), tokens.cpu().numpy(), logp.cpu().numpy()


def check_draw(z, u, rows=None, most_near=0.02, of=None, **kw):
    """`of`: the call's rows and numbers, and which of them z and u are."""
    settings = {k: kw[k] for k in ("temperature", "top_k", "top_p", "min_p") if k in kw}
    if of is None:
        x, tokens, logp = draw(z, u, rows=rows, **kw)
    else:
        x, tokens, logp = (r[of[2]] for r in draw(of[0], of[1], rows=rows, **kw))
    close = 0
    for t in range(len(z)):
        own = {k: float(np.float32(v)) for k, v in settings.items()}
        own.update({k: (v if of is None else v[of[2]])[t] for k, v in (rows or {}).items()})
        tok, lp, near = to.sample_row(x[t], np.float32(u[t]), **own)
        if near < NEAR:
            close += 1
            continue
        assert tokens[t] == tok, (t, own, u[t], near)
        if np.isinf(lp):
            assert logp[t] == lp
        else:
            V = len(z[t])
            cut = V * 2.0 ** (np.ceil(np.log2(V)) - 62) + 2.0 ** -50
            assert abs(logp[t] - lp) <= 2.0 ** -20 * abs(lp) + cut, (t, own, logp[t], lp)
    assert close <= 1 + most_near * len(z)
    return tokens


SETTINGS = [dict(), dict(temperature=0.7, top_k=20, top_p=0.8), dict(top_p=0.9), dict(top_k=50),
            dict(top_p=0.95, min_p=0.05), dict(top_p=0.99, min_p=0.5),
            dict(min_p=0.05), dict(top_k=300, min_p=0.01, temperature=1.7), dict(top_k=1),
            dict(temperature=0.0, top_p=0.5), dict(top_p=0.0), dict(top_k=7, top_p=0.99, min_p=0.2)]


@pytest.mark.parametrize("settings", SETTINGS, ids=str)
@pytest.mark.parametrize("T,V,dtype", [(1, 1, "f32"), (5, 2, "bf16"), (3, 7, "f32"), (9, 64, "bf16"),
                                       (40, 1000, "f32"), (17, 4099, "bf16"), (170, 5000, "f32"),
                                       (6, 32003, "bf16"), (3, 151936, "f32"),
                                       (2, 151936, "bf16"), (2, 262144, "f32"), (1, 390001, "f32"),
                                       (1, 780001, "bf16")])
def test_sample(T, V, dtype, settings):
    rng = np.random.default_rng(T * V + len(settings))
    check_draw(_rows(rng, T, V, "zipf"), rng.uniform(size=T), dtype=dtype, **settings)


@pytest.mark.parametrize("kind", ["flat", "wide", "equal", "few", "low"])
@pytest.mark.parametrize("settings", [dict(), dict(top_p=0.6), dict(top_k=2500, top_p=0.5),
                                      dict(top_k=1000), dict(top_k=30, top_p=0.7),
                                      dict(temperature=8.0, top_p=0.95), dict(min_p=1.0),
                                      dict(temperature=0.01)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_flat_and_tied(kind, settings, dtype):
    """Nuclei that no list holds, and borders among equal logits."""
    rng = np.random.default_rng(len(kind))
    for T, V in ((4, 9000), (2, 70001)):
        # (equal logits: the mass up to a border is a whole number of weights, and so exact)
        u = (rng.integers(0, V, T) + 0.5) / V
        check_draw(_rows(rng, T, V, kind), u, dtype=dtype, **settings)


def test_sample_ties_go_to_the_lowest_ids():
    z = np.zeros((3, 8192))
    u = np.array([0.0, 0.5, 1 - 2.0 ** -24])
    assert list(check_draw(z, u, top_k=4)) == [0, 2, 3]
    assert list(check_draw(z, u, top_p=0.25)) == [0, 1024, 2047]
    assert list(check_draw(z, u, top_k=4096)) == [0, 2048, 4095]
    assert list(check_draw(z, u, top_k=1)) == [0, 0, 0]
    z[:, 100] = -0.0
    assert list(check_draw(z, u, top_k=101)) == [0, 50, 100]
    z[:, 5000:5003] = 1.0
    assert list(check_draw(z, u, top_k=2)) == [5000, 5001, 5001]


@pytest.mark.parametrize("V", [5, 3000, 60000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_masked_rows(V, dtype):
    rng = np.random.default_rng(V)
    z = _rows(rng, 8, V, "flat")
    z[0] = -INF                                        # nothing left
    z[1] = np.nan
    z[2] = -INF
    z[2, V // 2] = -3.0                                # one left
    z[3, ::2] = np.nan
    z[4, 1:] = np.finfo(np.float32).min                # masks of the type's lowest value
    z[5, [0, V - 1]] = INF                             # infinities, all alike
    z[6, :V // 2] = -INF
    z[7] = np.finfo(np.float32).min
    u = rng.uniform(size=8)
    for settings in (dict(), dict(top_k=3), dict(top_p=0.5), dict(top_k=4, top_p=0.3, min_p=0.1),
                     dict(temperature=0.0)):
        tokens = check_draw(z, u, dtype=dtype, **settings)
        assert tokens[0] == tokens[1] == -1 and tokens[2] == V // 2 and tokens[5] in (0, V - 1)


def test_sample_odd_settings():
    rng = np.random.default_rng(3)
    T, V = 12, 500
    z = _rows(rng, T, V, "zipf")
    u = np.array([-1.0, np.nan, 0.0, 1.0, 2.0, 1 - 2.0 ** -24, 1e-30, 0.3, 0.5, 0.7, 0.9, 0.99])
    for settings in (dict(), dict(temperature=1e-38), dict(temperature=1e38), dict(temperature=INF),
                     dict(top_k=V), dict(top_k=V + 5), dict(top_k=-3), dict(top_p=7.0),
                     dict(min_p=-1.0), dict(min_p=9.0), dict(temperature=-1.0)):
        check_draw(z, u, **settings)


def test_sample_settings_of_rows():
    rng = np.random.default_rng(4)
    T, V = 64, 3001
    rows = dict(temperature=rng.choice([0.0, 0.5, 1.0, 2.0], T).astype(np.float32),
                top_k=rng.choice([0, 1, 5, 4000, 1500], T).astype(np.int32),
                top_p=rng.choice([0.0, 0.4, 0.9, 1.0], T).astype(np.float32),
                min_p=rng.choice([0.0, 0.1], T).astype(np.float32))
    rows["temperature"][3] = np.nan
    z, u = _rows(rng, T, V, "zipf"), rng.uniform(size=T)
    for dtype in ("f32", "bf16"):
        check_draw(z, u, rows=rows, dtype=dtype)
        check_draw(z, u, rows={"top_p": rows["top_p"]}, dtype=dtype, temperature=0.8)


@pytest.mark.parametrize("pad,lead", [(0, 0), (1, 0), (3, 1), (64, 7), (5, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_rows_apart(pad, lead, dtype):
    """Rows at every alignment; what lies between them is not read."""
    rng = np.random.default_rng(pad)
    for T, V in ((5, 1), (7, 13), (4, 5001), (2, 40000)):
        z, u = _rows(rng, T, V, "zipf"), rng.uniform(size=T)
        check_draw(z, u, dtype=dtype, pad=pad, lead=lead, top_p=0.9)
        check_draw(z, u, dtype=dtype, pad=pad, lead=lead)


def _many(rng, T, V, kind, some=9):
    """Rows that are read by one CTA each: `some` different ones, over and over."""
    return np.tile(_rows(rng, some, V, kind), (T // some + 1, 1))[:T]


@pytest.mark.parametrize("settings", SETTINGS + [dict(top_k=200), dict(top_k=250, top_p=0.9)], ids=str)
@pytest.mark.parametrize("T,V,dtype", [(64, 22001, "f32"), (64, 43003, "bf16"), (70, 49999, "f32"),
                                       (66, 60001, "f32"), (64, 100003, "bf16"), (65, 151936, "bf16"),
                                       (200, 50001, "f32")])
def test_sample_many_long_rows(T, V, dtype, settings):
    rng = np.random.default_rng(V + len(settings))
    z, u = _many(rng, T, V, "zipf"), rng.uniform(size=T)
    check_draw(z[::7], u[::7], of=(z, u, slice(None, None, 7)), dtype=dtype, pad=1, **settings)


@pytest.mark.parametrize("kind", ["flat", "wide", "equal", "few", "low"])
@pytest.mark.parametrize("settings", [dict(), dict(top_p=0.6), dict(top_k=2500, top_p=0.5),
                                      dict(top_k=30, top_p=0.7), dict(temperature=8.0, top_p=0.95),
                                      dict(min_p=1.0), dict(temperature=0.01),
                                      dict(top_p=0.9, min_p=0.5)], ids=str)
@pytest.mark.parametrize("V,dtype", [(60001, "f32"), (100003, "bf16")])
def test_sample_many_flat_and_tied_rows(kind, settings, V, dtype):
    rng = np.random.default_rng(len(kind))
    for T in (64, 160):                                # (one CTA a SM, two)
        z, u = _many(rng, T, V, kind), (rng.integers(0, V, T) + 0.5) / V
        check_draw(z[::19], u[::19], of=(z, u, slice(None, None, 19)), dtype=dtype, **settings)


@pytest.mark.parametrize("T", [66, 700])
@pytest.mark.parametrize("dtype,V", [("f32", 50001), ("bf16", 100003)])
def test_sample_many_rows_of_different_settings(T, dtype, V):
    rng = np.random.default_rng(T)
    rows = dict(temperature=rng.choice([0.0, 0.7, 1.0, 2.0], T).astype(np.float32),
                top_k=rng.choice([0, 1, 20, 300, V + 1], T).astype(np.int32),
                top_p=rng.choice([0.5, 0.95, 1.0], T).astype(np.float32),
                min_p=rng.choice([0.0, 0.1], T).astype(np.float32))
    z, u, at = _many(rng, T, V, "zipf"), rng.uniform(size=T), slice(None, None, T // 33)
    x, tokens, logp = draw(z, u, dtype, rows=rows)
    assert np.all((tokens >= 0) & (tokens < V)) and np.all(logp <= 0)
    check_draw(z[at], u[at], of=(z, u, at), dtype=dtype, rows=rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_many_masked_rows(dtype):
    """What the first ninth of a row shows says nothing of the rest."""
    rng = np.random.default_rng(11)
    T, V = 64, 110001
    z = _many(rng, T, V, "zipf", 16)
    z[0] = -INF
    z[1] = np.nan
    z[2] = -INF
    z[2, V - 1] = 2.0                                  # only the last is left
    z[3, :V - 5] = -INF                                # only the last five
    z[4, :V // 2] = np.nan
    z[5, 90000] = INF
    z[6] = np.arange(V) * 1e-3                         # rising: every part has a larger one
    z[7] = -np.arange(V) * 1e-3
    z[8] = np.finfo(np.float32).min
    z[9, 1000:] -= 200.0                               # all of it in the first share
    z[10, 7000::7] = -INF
    u = rng.uniform(size=T)
    for settings in (dict(), dict(top_k=3), dict(top_p=0.5), dict(top_k=40, top_p=0.3, min_p=0.1),
                     dict(temperature=0.0), dict(temperature=3.0, top_p=0.9), dict(min_p=0.3)):
        check_draw(z[:12], u[:12], of=(z, u, slice(0, 12)), dtype=dtype, **settings)
    check_top(z[:64], 40, dtype, rows=range(12))
    check_top(z[:64], 300, dtype, rows=range(12), lse=False)


@pytest.mark.parametrize("k", [1, 64, 256, 1000])
@pytest.mark.parametrize("V,dtype", [(25000, "f32"), (60001, "f32"), (100003, "bf16")])
def test_top_logits_many_long_rows(V, dtype, k):
    rng = np.random.default_rng(k)
    check_top(_many(rng, 65, V, "zipf"), k, dtype, pad=3, rows=range(0, 65, 9))
    check_top(_many(rng, 64, V, "few"), k, dtype, rows=range(0, 64, 20))


@pytest.mark.parametrize("dtype,V", [("f32", 500_001), ("bf16", 900_007)])
def test_sample_rows_that_no_cluster_holds(dtype, V):
    rng = np.random.default_rng(5)
    z, u = _rows(rng, 2, V, "zipf"), rng.uniform(size=2)
    for settings in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.99), dict(temperature=0.0)):
        check_draw(z, u, dtype=dtype, **settings)


def check_top(z, k, dtype="f32", pad=0, lead=0, lse=True, rows=None):
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V = z.shape
    x = _tensor(z, dtype, pad, lead)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    values = torch.full((T, k), 7.0, device="cuda")
    sums = torch.full((T,), 7.0, device="cuda") if lse else None
    tio.top_logits(x, ids, values, lse=sums)
    torch.cuda.synchronize()
    x = x.double().cpu().numpy()
    for t in range(T) if rows is None else rows:
        i, v, s = to.top_row(x[t], k)
        assert np.array_equal(ids[t].cpu().numpy(), i)
        assert np.array_equal(values[t].double().cpu().numpy(), v)
        if not lse:
            continue
        if not np.isfinite(s):
            assert float(sums[t]) == s
            continue
        # a term's exponent is rounded three times, the exponential is off by 2^-22 of itself;
        # a thread adds at most V / 512 terms; the maximum and the logarithm are added
        on = np.isfinite(x[t])
        p = np.exp(x[t][on] - s)
        away = np.sum(p * np.abs(x[t][on] - np.max(x[t][on])))
        bound = 2.0 ** -22 + 3 * 2.0 ** -24 * away + 2.0 ** -24 * (V / 512 + 40)
        assert abs(float(sums[t]) - s) <= bound + 2.0 ** -22 * abs(s) + 2.0 ** -22, (t, s)


@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 5, 5), (7, 64, 8), (33, 1000, 64), (200, 2049, 1),
                                   (5, 9001, 1024), (16, 32003, 33), (2, 151936, 8),
                                   (2, 151936, 256), (1, 600_001, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_top_logits(T, V, k, dtype):
    rng = np.random.default_rng(V)
    check_top(_rows(rng, T, V, "zipf"), k, dtype)
    check_top(_rows(rng, T, V, "flat"), k, dtype, pad=3, lead=1, lse=False)


@pytest.mark.parametrize("kind", ["wide", "equal", "few", "low"])
@pytest.mark.parametrize("k", [1, 40, 1000])
def test_top_logits_tied(kind, k):
    rng = np.random.default_rng(k)
    for dtype in ("f32", "bf16"):
        for V in (1500, 9000, 70001):
            check_top(_rows(rng, 3, V, kind), k, dtype)


def test_top_logits_masked():
    rng = np.random.default_rng(9)
    for V in (40, 5000):
        z = _rows(rng, 6, V, "flat")
        z[0] = -INF
        z[1, 3:] = -INF
        z[2, ::2] = np.nan
        z[3, 7] = INF
        z[4, 5:] = np.finfo(np.float32).min
        z[5] = np.nan
        check_top(z, 33)
        check_top(z, 33, "bf16")


def _embed(T, V, H, dtype, scale, ids):
    from dspark_block_drafter_gb300 import torch_io as tio
    g = torch.Generator(device="cuda").manual_seed(T + H)
    table = torch.randn(V, H, generator=g, device="cuda").to(DT[dtype])
    cfg = tio.make_embed_config(T, V, H, dtype, scale=scale)
    out = torch.full((T, H), 7.0, dtype=DT[dtype], device="cuda")
    tio.embed(cfg, table, torch.from_numpy(ids).cuda(), out)
    want = to.embed(table.double().cpu().numpy(), ids, np.float32(scale))
    # (the product is rounded to fp32 before bf16)
    bound = (OUT[dtype] + 2.0 ** -24) * np.abs(want) * (1 + 2.0 ** -8)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
    if scale == 1.0:
        assert np.array_equal(out.double().cpu().numpy(), want)


def _ids(rng, T, V, kind="skewed"):
    ids = (rng.uniform(size=T) ** 4 * V).astype(np.int32)
    if kind == "one":
        ids[:] = V - 1
    if kind == "all":
        ids = np.resize(rng.permutation(V), T).astype(np.int32)
    if kind == "none":
        ids[:] = -1
    return ids


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (16, 500, 4096), (3, 7, 5), (1000, 300, 64),
                                   (4999, 97, 1001), (5000, 400, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 53.25, 0.1])
def test_embed(T, V, H, dtype, scale):
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, V)
    ids[rng.uniform(size=T) < 0.1] = -1
    if T > 2:
        ids[1] = V
        ids[2] = 2 ** 31 - 1
    _embed(T, V, H, dtype, scale, ids)


def grad(T, V, H, dtype, scale=1.0, add=None, ids=None, kind="skewed", seed=0):
    from dspark_block_drafter_gb300 import torch_io as tio
    rng = np.random.default_rng(seed + T)
    if ids is None:
        ids = _ids(rng, T, V, kind)
    d = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).cuda().to(DT[dtype])
    # rows without a token are not read
    d[torch.from_numpy((ids < 0) | (ids >= V)).cuda()] = float("nan")
    base = None
    if add is not None:
        base = torch.from_numpy(rng.normal(size=(V, H)).astype(np.float32)).cuda().to(DT[dtype])
    table = base.clone() if add == "same" else torch.full((V, H), 7.0, dtype=DT[dtype],
                                                          device="cuda")
    cfg = tio.make_embed_config(T, V, H, dtype, scale=scale)
    ws = tio.embed_workspace_for(cfg)
    ws.fill_(0xFF)
    args = (cfg, torch.from_numpy(ids).cuda(), d, table, ws)
    tio.embed_backward(*args, add=table if add == "same" else base)
    torch.cuda.synchronize()
    assert tio.device_status(ws) == (5 if (ids >= V).any() else 0)
    dd = np.nan_to_num(d.double().cpu().numpy())
    want, mag = to.embed_backward(ids, dd, V, np.float32(scale),
                                  None if base is None else base.double().cpu().numpy())
    # fp32 sums in parts of a chunk, joined with their errors; scaled and added in one rounding
    chunk = max(32, (T + 2431) // 2432)
    bound = OUT[dtype] * np.abs(want) + (chunk + 4) * 2.0 ** -24 * mag * (1 + OUT[dtype])
    got = table.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound + 1e-30), np.max(np.abs(got - want) - bound)
    if add == "same":                      # rows that do not occur are left as they are
        off = np.setdiff1d(np.arange(V), ids)
        assert np.array_equal(got[off], base.double().cpu().numpy()[off])
    return args, got


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (2, 9, 8), (33, 5, 24), (100, 4000, 72), (1024, 64, 40),
                                   (1025, 300, 64), (4097, 1000, 33), (16384, 5000, 16),
                                   (16385, 5000, 16), (50000, 70000, 8), (300, 200, 5000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("add", [None, "other", "same"])
def test_embed_backward(T, V, H, dtype, add):
    grad(T, V, H, dtype, add=add)


@pytest.mark.parametrize("lead", [1, 3, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_backward_alignments(dtype, lead):
    """`add` and the table at different places within 16 bytes."""
    from dspark_block_drafter_gb300 import torch_io as tio
    T, V, H = 40, 300, 64
    g = torch.Generator(device="cuda").manual_seed(lead)
    ids = torch.randint(V, (T,), generator=g, device="cuda").int()
    flat = [torch.randn(n * H + lead, generator=g, device="cuda").to(DT[dtype]) for n in (V, V, T)]
    for moved in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)):
        add, table, d = (f[lead * m:lead * m + n * H].view(n, H)
                         for f, m, n in zip(flat, moved, (V, V, T)))
        cfg = tio.make_embed_config(T, V, H, dtype)
        tio.embed_backward(cfg, ids, d, table, tio.embed_workspace_for(cfg), add=add)
        want, mag = to.embed_backward(ids.cpu().numpy(), d.double().cpu().numpy(), V, 1.0,
                                      add.double().cpu().numpy())
        bound = OUT[dtype] * np.abs(want) + 36 * 2.0 ** -24 * mag * (1 + OUT[dtype])
        assert np.all(np.abs(table.double().cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("kind", ["one", "all", "none"])
@pytest.mark.parametrize("T,V", [(31, 40), (64, 64), (5000, 77), (20000, 700), (300_000, 1000)])
def test_embed_backward_tokens(kind, T, V):
    """One token in every row (joined over all chunks), every token, no token."""
    grad(T, V, 24, "f32", kind=kind, scale=0.5)
    grad(T, V, 24, "bf16", kind=kind, add="same")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [50, 100, 5000])
def test_embed_backward_infinities(T, dtype):
    """A sum with an infinity is that infinity, in one chunk or over many; inf - inf is NaN."""
    from dspark_block_drafter_gb300 import torch_io as tio
    H = 8
    d = torch.ones(T, H, device="cuda", dtype=DT[dtype])
    d[T // 3, 1] = d[T // 2, 2] = d[T // 3, 3] = float("inf")
    d[T // 2, 3] = d[T - 1, 4] = float("-inf")
    d[0, 5] = float("nan")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    table = torch.empty(3, H, device="cuda", dtype=DT[dtype])
    cfg = tio.make_embed_config(T, 3, H, dtype)
    tio.embed_backward(cfg, ids, d, table, tio.embed_workspace_for(cfg))
    want = d.double().sum(0).to(DT[dtype])
    assert torch.allclose(table[0], want, rtol=0, atol=0, equal_nan=True)
    assert not table[1:].any()


@pytest.mark.parametrize("T", [100, 20000])
def test_embed_backward_tokens_outside(T):
    rng = np.random.default_rng(1)
    ids = _ids(rng, T, 50)
    ids[::3] = -5
    grad(T, 50, 16, "f32", ids=ids.copy())
    ids[1::7] = 50
    ids[2::7] = 2 ** 31 - 1
    grad(T, 50, 16, "f32", ids=ids)
