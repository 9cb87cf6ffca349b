"""The operators on tokens and the distillation without a GPU: refusals come before any launch."""
import ctypes

import pytest
import torch

import dspark_block_drafter_gb300 as ds
from dspark_block_drafter_gb300 import _abi, torch_io as tio

I, U, W = _abi.DSPARK_ERR_INVALID_ARG, _abi.DSPARK_ERR_UNSUPPORTED, _abi.DSPARK_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(_abi.LIB_PATH):
        from dspark_block_drafter_gb300 import build
        build.build()
    return ds.lib()


def test_struct_layouts_match_c():
    assert ctypes.sizeof(_abi.dspark_teacher) == 32
    assert ctypes.sizeof(_abi.dspark_sample_config) == 40
    assert ctypes.sizeof(_abi.dspark_sample_rows) == 32
    assert ctypes.sizeof(_abi.dspark_embed_config) == 20


def _sample(logits=0x1000, uniform=0x2000, tokens=0x3000, logp=None, rows=None, **kw):
    c = dict(T=4, V=100, ld=100, dtype=0, top_k=0, temperature=1.0, top_p=1.0, min_p=0.0)
    c.update(kw)
    return ds.dspark_sample(_abi.dspark_sample_config(**c), rows, logits, uniform, tokens, logp)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), I), (dict(V=0), I), (dict(ld=99), I), (dict(dtype=2), I), (dict(dtype=-1), I),
    (dict(temperature=NAN), I), (dict(top_p=NAN), I), (dict(min_p=NAN), I),
    (dict(T=(1 << 20) + 1), U), (dict(V=(1 << 24) + 1, ld=1 << 25), U), (dict(ld=(1 << 32) + 1), U),
    (dict(logits=None), I), (dict(uniform=None), I), (dict(tokens=None), I),
    (dict(logits=0x1002), I), (dict(logits=0x1001, dtype=1), I), (dict(uniform=0x2002), I),
    (dict(tokens=0x3001), I), (dict(logp=0x4002), I),
    (dict(rows=_abi.dspark_sample_rows(top_k=0x5002)), I),
    (dict(rows=_abi.dspark_sample_rows(top_p=0x5001)), I),
    # (rows of logits: 0x1000 to 0x1640)
    (dict(tokens=0x1000), I), (dict(tokens=0x163C), I), (dict(logp=0xFF4), I), (dict(tokens=0x200C), I),
    (dict(logp=0x3000), I), (dict(logp=0x5000, rows=_abi.dspark_sample_rows(temperature=0x5000)), I),
    (dict(tokens=0x5004, rows=_abi.dspark_sample_rows(top_k=0x5000)), I)])
def test_sample_refusals(kw, status):
    assert _sample(**kw) == status
    assert ds.dspark_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), I), (dict(V=0), I), (dict(ld=99), I), (dict(dtype=3), I), (dict(k=0), I),
    (dict(k=101), I), (dict(k=1025, V=2000, ld=2000), U), (dict(T=(1 << 20) + 1), U),
    (dict(logits=None), I), (dict(ids=None), I), (dict(values=None), I), (dict(ids=0x2002), I),
    (dict(lse=0x4001), I), (dict(logits=0x1001, dtype=1), I), (dict(ids=0x163C), I),
    (dict(values=0x204C), I), (dict(lse=0x304C), I), (dict(lse=0x1000), I)])
def test_top_logits_refusals(kw, status):
    c = dict(T=4, V=100, ld=100, dtype=0, k=5, logits=0x1000, ids=0x2000, values=0x3000, lse=None)
    c.update(kw)
    assert ds.dspark_top_logits(**c) == status
    assert ds.dspark_last_error()


def _embed(**kw):
    c = dict(T=4, V=100, H=64, dtype=0, scale=1.0)
    c.update(kw)
    return _abi.dspark_embed_config(**c)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), I), (dict(V=0), I), (dict(H=0), I), (dict(dtype=2), I), (dict(scale=NAN), I),
    (dict(scale=INF), I), (dict(T=(1 << 20) + 1), U), (dict(V=(1 << 24) + 1), U),
    (dict(H=(1 << 16) + 1), U)])
def test_embed_refusals(kw, status):
    c = _embed(**kw)
    assert ds.dspark_embed(c, 0x100000, 0x2000, 0x3000) == status
    assert ds.dspark_embed_workspace_size(c) == 0
    assert ds.dspark_embed_backward(c, 0x2000, 0x3000, None, 0x100000, 0x1000000, 1 << 40) == status


def test_embed_call_refusals():
    c = _embed()
    # (a table of 25600 bytes, rows of 1024)
    for args in ((None, 0x2000, 0x3000), (0x100000, None, 0x3000), (0x100000, 0x2000, None),
                 (0x100002, 0x2000, 0x3000), (0x100000, 0x2001, 0x3000),
                 (0x100000, 0x2000, 0x100000), (0x100000, 0x2000, 0x100000 + 25600 - 4),
                 (0x100000, 0x2000, 0x100000 - 1024 + 4), (0x100000, 0x2000, 0x200C)):
        assert ds.dspark_embed(c, *args) == I, args
    need = ds.dspark_embed_workspace_size(c)
    assert need > 0 and need % 256 == 0
    ok = [0x2000, 0x3000, None, 0x100000, 0x1000000, need]
    for at, value, status in ((0, None, I), (1, None, I), (3, None, I), (0, 0x2002, I), (1, 0x3002, I),
                              (2, 0x200002, I), (3, 0x100001, I), (4, None, W), (4, 0x1000010, W),
                              (5, need - 1, W), (1, 0x100000, I), (1, 0x100000 + 25600 - 4, I),
                              (2, 0x100004, I), (2, 0x100000 - 25600 + 4, I), (0, 0x100004, I)):
        args = list(ok)
        args[at] = value
        assert ds.dspark_embed_backward(c, *args) == status, (at, value)


def test_embed_workspace_stays_small():
    """A share of the rows, whatever the table's size."""
    for T in (1, 1000, 16384, 1 << 20):
        n = ds.dspark_embed_workspace_size(_embed(T=T, V=1 << 18, H=4096, dtype=1))
        assert n < (1 << 17) + 64 * T + 4 * 2 * 4096 * (2432 + T // 32 if T < 77824 else 2432) + (1 << 22)


def _cfg(**kw):
    c = dict(T=5, H=64, V=1000, r=8, dtype=0, reduction=1, vocab_pieces=0, loss_scale=1.0)
    c.update(kw)
    return _abi.dspark_loss_config(**c)


def _distill(cfg=None, teacher=None, head=None, out=None, hidden=0x4000, prev=0x5000, weights=None,
             ws=0x10000, n=None):
    c = _cfg(**(cfg or {}))
    t = dict(ids=0x6000, logits=0x7000, lse=None, k=8, scale=1.0)
    t.update(teacher or {})
    h = dict(lm_head=0x1000, V_head=1000, markov_w1=0x2000, markov_w2=0x3000)
    h.update(head or {})
    o = dict(loss=0x100, total=0x200)
    o.update(out or {})
    h, t, o = _abi.dspark_head(**h), _abi.dspark_teacher(**t), _abi.dspark_loss_outputs(**o)
    need = ds.dspark_distill_loss_workspace_size(c, h, t, o)
    return need, ds.dspark_distill_loss(c, h, hidden, prev, t, weights, o, ws,
                                        need if n is None else n)


@pytest.mark.parametrize("kw,status", [
    (dict(cfg=dict(T=0)), I), (dict(cfg=dict(dtype=5)), I), (dict(cfg=dict(r=513)), U),
    (dict(cfg=dict(loss_scale=NAN)), I), (dict(teacher=dict(k=0)), I), (dict(teacher=dict(k=-1)), I),
    (dict(teacher=dict(k=257)), U), (dict(teacher=dict(scale=INF)), I), (dict(teacher=dict(scale=NAN)), I),
    (dict(head=dict(lm_head=None)), I), (dict(head=dict(markov_w1=None)), I)])
def test_distill_refusals(kw, status):
    assert _distill(**kw, n=1 << 40) == (0, status)
    assert ds.dspark_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(teacher=dict(ids=None)), I), (dict(teacher=dict(logits=None)), I),
    (dict(teacher=dict(ids=0x6002)), I), (dict(teacher=dict(logits=0x7001)), I),
    (dict(teacher=dict(lse=0x8002)), I), (dict(hidden=None), I), (dict(prev=None), I),
    (dict(weights=0x9001), I), (dict(out=dict(loss=None)), I), (dict(out=dict(total=None)), I),
    (dict(ws=None), W), (dict(ws=0x10010), W), (dict(n=100), W)])
def test_distill_call_refusals(kw, status):
    need, st = _distill(**kw)
    assert need > 0 and st == status


def test_distill_workspace_is_the_head_loss_s_and_the_lists():
    for T, k in ((5, 8), (4096, 64)):
        c = _cfg(T=T)
        h = _abi.dspark_head(lm_head=0x1000, V_head=1000, markov_w1=0x2000, markov_w2=0x3000)
        o = _abi.dspark_loss_outputs(loss=0x100, total=0x200, d_hidden=0x300)
        t = _abi.dspark_teacher(ids=0x6000, logits=0x7000, k=k, scale=1.0)
        more = (ds.dspark_distill_loss_workspace_size(c, h, t, o)
                - ds.dspark_head_loss_workspace_size(c, h, o))
        assert 12 * T * k <= more <= 12 * (T + 256) * k + 16 * (T + 256) + 6 * 256


def test_null_structs_are_refused():
    lib = ds.lib()
    assert lib.dspark_sample(None, None, 1 << 12, 1 << 13, 1 << 14, None, 0) == I
    assert lib.dspark_embed(None, 1 << 12, 1 << 13, 1 << 14, 0) == I
    assert lib.dspark_embed_workspace_size(None) == 0
    assert lib.dspark_embed_backward(None, 16, 16, None, 16, 256, 1 << 20, 0) == I
    c, h, o = _cfg(), _abi.dspark_head(lm_head=16, V_head=1000, markov_w1=16, markov_w2=16), \
        _abi.dspark_loss_outputs(loss=16, total=16)
    assert lib.dspark_distill_loss_workspace_size(ctypes.byref(c), ctypes.byref(h), None,
                                                  ctypes.byref(o)) == 0
    assert lib.dspark_distill_loss(ctypes.byref(c), ctypes.byref(h), 16, 16, None, None,
                                   ctypes.byref(o), 256, 1 << 30, 0) == I


# ------------------------------------------------------------------ the torch calls' own checks
def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(logits=_z(3, 10)), dict(logits=_z(4, 10, dtype=torch.bfloat16)), dict(logits=_z(10, 4).t()),
    dict(logits=_z(1, 10).expand(4, 10)), dict(logits=_z(40)), dict(uniform=_z(3)),
    dict(uniform=_z(4, dtype=torch.float64)), dict(tokens=_z(4)), dict(tokens=_z(8, dtype=torch.int32)[::2]),
    dict(logp=_z(5)), dict(top_k=_z(4)), dict(top_k=_z(4, dtype=torch.int64)),
    dict(temperature=_z(3)), dict(top_p=_z(4, 1)), dict(min_p=_z(4, dtype=torch.bfloat16))])
def test_sample_checks_its_tensors(kw):
    a = dict(logits=_z(4, 10), uniform=_z(4), tokens=_z(4, dtype=torch.int32))
    a.update(kw)
    with pytest.raises(ValueError):
        tio.sample(tio.make_sample_config(4, 10, "f32"), a.pop("logits"), a.pop("uniform"),
                   a.pop("tokens"), **a)


def test_cpu_tensors_are_refused():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="current GPU"):
        tio.sample(tio.make_sample_config(4, 10, "f32"), _z(4, 10), _z(4), _z(4, **i32))
    with pytest.raises(ValueError, match="current GPU"):
        tio.top_logits(_z(4, 10), _z(4, 2, **i32), _z(4, 2))
    with pytest.raises(ValueError, match="current GPU"):
        tio.embed(tio.make_embed_config(4, 10, 8, "f32"), _z(10, 8), _z(4, **i32), _z(4, 8))
    with pytest.raises(ValueError, match="current GPU"):
        tio.embed_backward(tio.make_embed_config(4, 10, 8, "f32"), _z(4, **i32), _z(4, 8), _z(10, 8),
                           _z(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("logits,ids,values,lse", [
    (_z(4, 10, dtype=torch.float16), _z(4, 2, dtype=torch.int32), _z(4, 2), None),
    (_z(4, 10), _z(4, 2, dtype=torch.int64), _z(4, 2), None),
    (_z(4, 10), _z(3, 2, dtype=torch.int32), _z(4, 2), None),
    (_z(4, 10), _z(4, 2, dtype=torch.int32), _z(4, 3), None),
    (_z(4, 10), _z(4, 2, dtype=torch.int32), _z(4, 2), _z(3)),
    (_z(4, 20)[:, ::2], _z(4, 2, dtype=torch.int32), _z(4, 2), None),
    (_z(40), _z(4, 2, dtype=torch.int32), _z(4, 2), None)])
def test_top_logits_checks_its_tensors(logits, ids, values, lse):
    with pytest.raises(ValueError):
        tio.top_logits(logits, ids, values, lse=lse)


def test_embed_and_distill_check_their_tensors():
    c, i32 = tio.make_embed_config(4, 10, 8, "bf16"), dict(dtype=torch.int32)
    b = dict(dtype=torch.bfloat16)
    for t, i, o in ((_z(10, 8), _z(4, **i32), _z(4, 8, **b)), (_z(9, 8, **b), _z(4, **i32), _z(4, 8, **b)),
                    (_z(10, 8, **b), _z(4), _z(4, 8, **b)), (_z(10, 8, **b), _z(4, **i32), _z(8, 4, **b).t())):
        with pytest.raises(ValueError):
            tio.embed(c, t, i, o)
    ws = _z(1 << 20, dtype=torch.uint8)
    for kw in (dict(d_out=_z(4, 8)), dict(d_table=_z(4, 8, **b)), dict(add=_z(10, 8))):
        a = dict(d_out=_z(4, 8, **b), d_table=_z(10, 8, **b), add=None)
        a.update(kw)
        with pytest.raises(ValueError):
            tio.embed_backward(c, _z(4, **i32), a["d_out"], a["d_table"], ws, add=a["add"])
    cfg = tio.make_loss_config(4, 8, 16, 0, "f32")
    head = tio.Head(_z(16, 8), None, None, None, None)
    out = tio.LossOutputs(_z(4), _z(1))
    for t in (tio.Teacher(_z(4, 3), _z(4, 3)), tio.Teacher(_z(4, 3, **i32), _z(4, 2)),
              tio.Teacher(_z(12, **i32), _z(12)), tio.Teacher(_z(4, 3, **i32), _z(4, 3), lse=_z(3))):
        with pytest.raises(ValueError):
            tio.distill_loss(cfg, head, t, _z(4, 8), None, out, ws)
