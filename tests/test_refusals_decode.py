"""Tables whose tiles the partial decodes could not count in 32 bits are refused before anything is launched (no GPU)."""

import ctypes

import pytest

import context_sharded_mla_gb300 as dcp

UNSUPPORTED = -2
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from context_sharded_mla_gb300 import _build
    _build.build()
    return dcp.load_library()


# The planner counts tiles of 64 rows over all units: B * 4 shards * max_pages * P / 64, a unit's rows capped at 2^30.
# One request in four shards: 2^31 - 256 rows at most in the pools, so the table repeats pages.
@pytest.mark.parametrize("page,max_pages,B", [
    (1 << 20, 1 << 12, 32),         # 4 Gi rows a unit, capped at 2^24 tiles: 128 units of them
    (64, 1 << 20, 512),             # 2^20 tiles a unit, 2048 units
    (64, 1 << 40, 32),
    (8, 1 << 62, 1 << 20),
])
@pytest.mark.parametrize("entry", ["dcp_mla_decode_partial", "dcp_mla_decode_partial_q4", "dcp_mla_decode_partial_static"])
def test_too_many_tiles(lib, entry, page, max_pages, B):
    lay = dcp.Layout(4, 1, page)
    args = [ctypes.byref(lay), 0, 4, P(256), B, 1, 1, P(256), 1, P(256), max_pages, max_pages, P(256), 0.1, 0, P(256), 0,
            P(256)]
    args += [P(256), None] if entry.endswith("static") else [None, 0, P(256), None]
    assert getattr(lib, entry)(*args) == UNSUPPORTED
