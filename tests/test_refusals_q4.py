"""What the 4-bit cache's calls and dcp_block_tables refuse, before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

import context_sharded_mla_gb300 as dcp
from context_sharded_mla_gb300.step import ShardedMlaDecoder

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -4
P = ctypes.c_void_p
GOOD, BAD, HUGE = dcp.Layout(4, 1, 16), dcp.Layout(4, 3, 16), 2 ** 62


@pytest.fixture(scope="module")
def lib():
    from context_sharded_mla_gb300 import _build
    _build.build()
    return dcp.load_library()


def call(fn, defaults, **kw):
    lay = kw.pop("lay", GOOD)
    assert not set(kw) - set(defaults)
    return fn(ctypes.byref(lay) if lay else None, *dict(defaults, **kw).values())


@pytest.mark.parametrize("kw", [
    dict(lay=None), dict(lay=BAD), dict(sb=-1), dict(se=5), dict(sb=2, se=2), dict(T=-1), dict(B=0), dict(mp=0),
    dict(mp=2), dict(pp=0), dict(kv=None), dict(kv=P(24)), dict(pos=None), dict(req=None), dict(bt=None), dict(ar=None),
    dict(ar=P(40))])
def test_append_and_read(lib, kw):
    base = dict(sb=0, se=4, kv=P(16), pos=P(16), req=P(16), T=1, bt=P(16), B=1, st=1, mp=1, ar=P(32), pp=1, status=P(16),
                stream=None)
    assert call(lib.dcp_kv_append_q4, base, **kw) == INVALID
    order = ("sb", "se", "ar", "pp", "pos", "req", "T", "bt", "B", "st", "mp", "kv", "status", "stream")
    assert call(lib.dcp_kv_read_q4, {k: base[k] for k in order}, **kw) == INVALID
    assert call(lib.dcp_kv_append_q4, base, T=0) == 0               # nothing to do, nothing launched
    assert call(lib.dcp_kv_read_q4, {k: base[k] for k in order}, T=0) == 0
    assert call(lib.dcp_kv_append_q4, base, T=HUGE) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(lay=BAD), dict(se=5), dict(src=None), dict(src=P(24)), dict(rows=0), dict(Ps=0), dict(sbt=None), dict(smp=0),
    dict(smp=2), dict(T=-1), dict(B=0), dict(mp=2), dict(pp=0), dict(pos=None), dict(req=None), dict(bt=None),
    dict(ar=None), dict(ar=P(40)), dict(status=None)])
def test_relayout(lib, kw):
    base = dict(sb=0, se=4, src=P(16), rows=8, Ps=8, sbt=P(16), sst=1, smp=1, pos=P(16), req=P(16), T=1, B=1, bt=P(16),
                st=1, mp=1, ar=P(32), pp=1, status=P(16), stream=None)
    assert call(lib.dcp_kv_relayout_q4, base, **kw) == INVALID
    assert call(lib.dcp_kv_relayout_q4, base, T=0) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=BAD), INVALID), (dict(se=5), INVALID), (dict(q=None), INVALID), (dict(q=P(264)), INVALID),
    (dict(B=0), INVALID), (dict(H=65537), INVALID), (dict(ql=512, H=129), INVALID), (dict(ar=None), INVALID),
    (dict(ar=P(264)), INVALID), (dict(pp=0), INVALID), (dict(bt=None), INVALID), (dict(mp=2), INVALID),
    (dict(sl=None), INVALID), (dict(sc=0.0), INVALID), (dict(sc=float("inf")), INVALID), (dict(sc=float("nan")), INVALID),
    (dict(base=7), INVALID), (dict(op=None), INVALID), (dict(op=P(264)), INVALID), (dict(od=9), INVALID),
    (dict(lp=None), INVALID), (dict(lay=dcp.Layout(4, 1, 12)), UNSUPPORTED), (dict(lay=dcp.Layout(4, 1, 4)), UNSUPPORTED),
    (dict(pp=2 ** 27), UNSUPPORTED)])
def test_partial(lib, kw, rc):
    base = dict(sb=0, se=4, q=P(256), B=1, ql=1, H=16, ar=P(256), pp=1, bt=P(256), st=1, mp=1, sl=P(256), sc=0.1, base=0,
                op=P(256), od=0, lp=P(256), ws=None, wsb=0, status=P(256), stream=None)
    assert call(lib.dcp_mla_decode_partial_q4, base, **kw) == rc
    need = lib.dcp_mla_decode_workspace_size_q4(ctypes.byref(GOOD), 0, 4, 1, 1, 16)   # 0 where there is no device
    if need:
        assert call(lib.dcp_mla_decode_partial_q4, base, ws=P(256), wsb=need - 1) == WORKSPACE
        assert call(lib.dcp_mla_decode_partial_q4, base, ws=P(264), wsb=need) == INVALID


def test_workspace_size_of_bad_arguments(lib):
    size = lib.dcp_mla_decode_workspace_size_q4
    for lay, *rest in ((BAD, 0, 4, 1, 1, 16), (GOOD, 0, 5, 1, 1, 16), (GOOD, 0, 4, 0, 1, 16), (GOOD, 0, 4, 1, 0, 16),
                       (GOOD, 0, 4, 1, 512, 129)):
        assert size(ctypes.byref(lay), *rest) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=None), INVALID), (dict(lay=BAD), INVALID), (dict(B=0), INVALID), (dict(seq=None), INVALID),
    (dict(new=None), INVALID), (dict(seq=P(48)), INVALID), (dict(bt=None), INVALID), (dict(mp=0), INVALID),
    (dict(mp=2), INVALID), (dict(free=None), INVALID), (dict(state=None), INVALID), (dict(pp=0), INVALID),
    (dict(pp=2 ** 31), INVALID), (dict(T=-1), INVALID), (dict(pos=None), INVALID), (dict(req=None), INVALID),
    (dict(pos=None, req=None), INVALID), (dict(cu=None), INVALID), (dict(status=None), INVALID),
    (dict(T=HUGE), UNSUPPORTED)])
def test_block_tables(lib, kw, rc):
    base = dict(B=1, seq=P(16), new=P(48), bt=P(16), st=1, mp=1, free=P(16), state=P(16), pp=1, T=1, pos=P(16), req=P(16),
                owner=P(16), row=P(16), slot=P(16), cu=P(16), status=P(16), stream=None)
    assert call(lib.dcp_block_tables, base, **kw) == rc


def test_unknown_cache_format():
    with pytest.raises(ValueError, match="cache format"):
        ShardedMlaDecoder(GOOD, 1, 1, 16, 4, 1, 0.1, device="cpu", cache="q2")


def test_tensors_that_are_not_on_the_gpu(monkeypatch):
    """The Python entry points name the first argument that cannot be used."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, d=torch.int64: torch.zeros(*s, dtype=d)
    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    arena, pos, req, bt, st = z(4, 16, 416, d=u8), z(2), z(2, d=i32), z(1, 1, d=i32), z(1, d=i32)
    with pytest.raises(ValueError, match="kv_new must be a CUDA tensor"):
        dcp.dcp_kv_append_q4(GOOD, 0, 4, z(2, 576, d=bf), pos, req, bt, 1, arena, 1, st)
    with pytest.raises(ValueError, match="arena must be a CUDA tensor"):
        dcp.dcp_kv_read_q4(GOOD, 0, 4, arena, 1, pos, req, bt, 1, z(2, 576, d=bf), st)
    with pytest.raises(ValueError, match="one row per request"):
        dcp.dcp_kv_relayout_q4(GOOD, 0, 4, z(8, 576, d=bf), 8, z(2, 1, d=i32), 1, pos, req, bt, 1, arena, 1, st)
    with pytest.raises(ValueError, match="src_pool must be"):
        dcp.dcp_kv_relayout_q4(GOOD, 0, 4, z(8, 512, d=bf), 8, z(1, 1, d=i32), 1, pos, req, bt, 1, arena, 1, st)
    with pytest.raises(ValueError, match="block_table must be"):
        dcp.dcp_kv_append_q4(GOOD, 0, 4, z(2, 576, d=bf), pos, req, z(1, d=i32), 1, arena, 1, st)
    o, lse = z(4, 1, 1, 16, 512, d=torch.float32), z(4, 1, 1, 16, d=torch.float32)
    with pytest.raises(ValueError, match="q must be"):
        dcp.dcp_mla_decode_partial_q4(GOOD, 0, 4, z(1, 16, 576, d=bf), arena, 1, bt, 1, z(1), 0.1, 0, o, lse, None, st)
    with pytest.raises(ValueError, match="one row per request"):
        dcp.dcp_mla_decode_partial_q4(GOOD, 0, 4, z(2, 1, 16, 576, d=bf), arena, 1, bt, 1, z(2), 0.1, 0, o, lse, None, st)
    with pytest.raises(ValueError, match="pos is empty"):
        dcp.dcp_block_tables(GOOD, z(1), z(1), bt, 1, z(1, d=i32), z(2), z(2), st, pos=z(0), req=z(0, d=i32))
    with pytest.raises(ValueError, match="pos must be a CUDA tensor"):
        dcp.dcp_block_tables(GOOD, z(1), z(1), bt, 1, z(1, d=i32), z(2), z(2), st, pos=z(3), req=z(3, d=i32))
