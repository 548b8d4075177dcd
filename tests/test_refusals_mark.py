"""What dcp_key_weights_mark refuses, before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

import context_sharded_mla_gb300 as dcp

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from context_sharded_mla_gb300 import _build
    _build.build()
    return dcp.load_library()


@pytest.mark.parametrize("kw,rc", [
    (dict(lay=None), INVALID), (dict(lay=dcp.Layout(4, 3, 16)), INVALID), (dict(sb=-1), INVALID), (dict(se=5), INVALID),
    (dict(sb=2, se=2), INVALID), (dict(B=0), INVALID), (dict(f=None), INVALID), (dict(s=None), INVALID),
    (dict(w=None), INVALID), (dict(ws=0), INVALID), (dict(B=2 ** 30), UNSUPPORTED)])
def test_mark(lib, kw, rc):
    base = dict(lay=dcp.Layout(4, 1, 16), sb=0, se=4, B=1, f=P(16), s=P(16), w=P(16), ws=16, stream=None)
    args = dict(base, **kw)
    lay = args.pop("lay")
    assert lib.dcp_key_weights_mark(ctypes.byref(lay) if lay else None, *args.values()) == rc


def test_tensors_that_cannot_be_used(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="from_lens must be a CUDA tensor"):
        dcp.dcp_key_weights_mark(dcp.Layout(4, 1, 16), 0, 4, z, z, torch.zeros(4, 1, 8))
