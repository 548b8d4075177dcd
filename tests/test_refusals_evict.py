"""What the norm/rotation, key-weight and eviction calls refuse, before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

import context_sharded_mla_gb300 as dcp

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -4
P = ctypes.c_void_p
GOOD, BAD, HUGE = dcp.Layout(4, 1, 16), dcp.Layout(4, 3, 16), 2 ** 62
NAN, INF = float("nan"), float("inf")


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
    dict(T=-1), dict(H=0), dict(H=65536), dict(q=None), dict(q=P(24)), dict(qs=191), dict(qs=196), dict(pos=None), dict(g=P(24)),
    dict(gd=2), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(style=2), dict(out=None), dict(out=P(40))])
def test_q_norm_rope(lib, kw):
    base = dict(T=1, H=2, q=P(16), qs=192, pos=P(16), g=P(16), gd=1, eps=1e-6, f=P(16), style=0, out=P(32), status=None,
                stream=None)
    assert lib.dcp_q_norm_rope(*dict(base, **kw).values()) == INVALID
    assert lib.dcp_q_norm_rope(*dict(base, T=0, q=None, out=None).values()) == 0
    assert lib.dcp_q_norm_rope(*dict(base, T=HUGE).values()) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(lay=None), dict(lay=BAD), dict(sb=-1), dict(se=5), dict(sb=2, se=2), dict(kv=None), dict(kv=P(24)), dict(ks=575),
    dict(ks=580), dict(g=P(24)), dict(gd=7), dict(eps=-0.5), dict(eps=NAN), dict(style=-1), dict(pos=None),
    dict(req=None), dict(T=-1), dict(bt=None), dict(B=0), dict(mp=0), dict(mp=2), dict(ar=None), dict(ar=P(40)),
    dict(pp=0)])
def test_norm_rope_append(lib, kw):
    base = dict(sb=0, se=4, kv=P(16), ks=576, g=P(16), gd=0, eps=0.0, f=P(16), style=1, rp=None, pos=P(16), req=P(16), T=1,
                bt=P(16), B=1, st=1, mp=1, ar=P(32), pp=1, status=P(16), stream=None)
    for fn in (lib.dcp_kv_norm_rope_append, lib.dcp_kv_norm_rope_append_q4):
        assert call(fn, base, **kw) == INVALID
        assert call(fn, base, T=0, kv=None) == 0
        assert call(fn, base, T=HUGE) == UNSUPPORTED


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=None), INVALID), (dict(lay=BAD), INVALID), (dict(se=5), INVALID), (dict(q=None), INVALID),
    (dict(q=P(264)), INVALID), (dict(B=0), INVALID), (dict(ql=0), INVALID), (dict(H=65537), INVALID),
    (dict(ql=512, H=129), INVALID), (dict(ar=None), INVALID), (dict(ar=P(264)), INVALID), (dict(pp=0), INVALID),
    (dict(bt=None), INVALID), (dict(mp=2), INVALID), (dict(sl=None), INVALID), (dict(sc=0.0), INVALID),
    (dict(sc=INF), INVALID), (dict(sc=NAN), INVALID), (dict(base=7), INVALID), (dict(lse=None), INVALID),
    (dict(decay=-0.1), INVALID), (dict(decay=NAN), INVALID), (dict(decay=INF), INVALID), (dict(w=None), INVALID),
    (dict(ws=15), INVALID), (dict(ws=-16), INVALID), (dict(lay=dcp.Layout(4, 1, 12)), UNSUPPORTED),
    (dict(lay=dcp.Layout(4, 1, 4)), UNSUPPORTED), (dict(pp=2 ** 27), UNSUPPORTED),
    (dict(B=2 ** 15, st=2 ** 22, mp=2 ** 22, ws=2 ** 40), UNSUPPORTED)])
def test_key_weights(lib, kw, rc):
    base = dict(sb=0, se=4, q=P(256), B=1, ql=1, H=16, ar=P(256), pp=1, bt=P(256), st=1, mp=1, sl=P(256), sc=0.1, base=0,
                lse=P(256), old=None, decay=1.0, w=P(256), ws=16, work=None, wb=0, status=P(256), stream=None)
    for fn in (lib.dcp_mla_key_weights, lib.dcp_mla_key_weights_q4):
        assert call(fn, base, **kw) == rc


def test_key_weights_workspace(lib):
    sizes = (lib.dcp_mla_key_weights_workspace_size, lib.dcp_mla_key_weights_workspace_size_q4)
    assert [f(4, 128) for f in sizes] == [f(0, 128) for f in sizes] == [f(2, -1) for f in sizes] == [0, 0]
    assert sizes[0](8, 128) == 0 < sizes[0](1025, 1) and 0 < sizes[1](513, 1)
    base = dict(sb=0, se=4, q=P(256), B=1, ql=1025, H=1, ar=P(256), pp=1, bt=P(256), st=1, mp=1, sl=P(256), sc=0.1,
                base=0, lse=P(256), old=None, decay=1.0, w=P(256), ws=16, work=P(256), wb=0, status=P(256), stream=None)
    for fn, size in zip((lib.dcp_mla_key_weights, lib.dcp_mla_key_weights_q4), sizes):
        assert call(fn, base, wb=size(1025, 1) - 1) == WORKSPACE
        assert call(fn, base, work=P(264), wb=size(1025, 1)) == INVALID


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=BAD), INVALID), (dict(se=5), INVALID), (dict(B=0), INVALID), (dict(sl=None), INVALID),
    (dict(nl=None), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(w=None), INVALID),
    (dict(ws=0), INVALID), (dict(k=None), INVALID), (dict(ks=0), INVALID), (dict(ws=2 ** 31), UNSUPPORTED),
    (dict(B=2 ** 30), UNSUPPORTED)])
def test_select(lib, kw, rc):
    base = dict(sb=0, se=4, B=1, sl=P(16), nl=P(16), sinks=0, recent=0, w=P(16), ws=16, k=P(16), ks=16, status=P(16),
                stream=None)
    assert call(lib.dcp_evict_select, base, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=BAD), INVALID), (dict(sb=3, se=3), INVALID), (dict(k=None), INVALID), (dict(ks=-1), INVALID),
    (dict(B=0), INVALID), (dict(nl=None), INVALID), (dict(bt=None), INVALID), (dict(mp=0), INVALID),
    (dict(mp=2), INVALID), (dict(ar=None), INVALID), (dict(ar=P(40)), INVALID), (dict(pp=0), INVALID),
    (dict(ws=0), INVALID), (dict(ks=2 ** 31), UNSUPPORTED), (dict(ks=0, k=None), 0)])
def test_compact(lib, kw, rc):
    base = dict(sb=0, se=4, k=P(16), ks=4, B=1, nl=P(16), bt=P(16), st=1, mp=1, ar=P(32), pp=1, w=P(16), ws=4,
                status=P(16), stream=None)
    for fn in (lib.dcp_kv_compact, lib.dcp_kv_compact_q4):
        assert call(fn, base, **kw) == rc


def test_tensors_that_cannot_be_used(lib, monkeypatch):
    """The Python entry points name the argument."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = lambda *s, d=torch.int64: torch.zeros(*s, dtype=d)   # noqa: E731
    i32, u8, bf, f32 = torch.int32, torch.uint8, torch.bfloat16, torch.float32
    arena, bt, st = z(4, 16, 576, d=bf), z(1, 1, d=i32), z(1, d=i32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dcp.dcp_q_norm_rope(z(2, 3, 192, d=bf), z(2), z(2, 3, 192, d=bf))
    with pytest.raises(ValueError, match="out must be"):
        dcp.dcp_q_norm_rope(z(2, 3, 192, d=bf), z(2), z(2, 576, d=bf))
    with pytest.raises(ValueError, match="kv must be a CUDA tensor"):
        dcp.dcp_kv_norm_rope_append(GOOD, 0, 4, z(2, 576, d=bf), z(2), z(2, d=i32), bt, 1, arena, 1, st)
    with pytest.raises(ValueError, match="block_table must be"):
        dcp.dcp_kv_norm_rope_append_q4(GOOD, 0, 4, z(2, 576, d=bf), z(2), z(2, d=i32), z(1, d=i32), 1, arena, 1, st)
    lse, w = z(1, 1, 16, d=f32), z(4, 1, 16, d=f32)
    with pytest.raises(ValueError, match="q must be"):
        dcp.dcp_mla_key_weights(GOOD, 0, 4, z(1, 16, 576, d=bf), arena, 1, bt, 1, z(1), 0.1, 0, lse, w, st)
    with pytest.raises(ValueError, match="one row per request"):
        dcp.dcp_mla_key_weights(GOOD, 0, 4, z(2, 1, 16, 576, d=bf), arena, 1, bt, 1, z(2), 0.1, 0, lse, w, st)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        dcp.dcp_mla_key_weights(GOOD, 0, 4, z(1, 1, 16, 576, d=bf), arena, 1, bt, 1, z(1), 0.1, 0, lse, w, st)
    with pytest.raises(ValueError, match="workspace must"):
        dcp.dcp_mla_key_weights(GOOD, 0, 4, z(1, 1, 16, 576, d=bf), arena, 1, bt, 1, z(1), 0.1, 0, lse, w, st, workspace=z(4))
    with pytest.raises(ValueError, match="seq_lens must be a CUDA tensor"):
        dcp.dcp_evict_select(GOOD, 0, 4, z(1), z(1), 0, 0, w, z(4, 1, 4, d=i32), st)
    with pytest.raises(ValueError, match="kept must"):
        dcp.dcp_kv_compact(GOOD, 0, 4, z(4, 2, 4, d=i32), z(1), bt, 1, arena, 1, st)
    with pytest.raises(ValueError, match="kept must be a CUDA tensor"):
        dcp.dcp_kv_compact_q4(GOOD, 0, 4, z(4, 1, 4, d=i32), z(1), bt, 1, z(4, 16, 416, d=u8), 1, st)
