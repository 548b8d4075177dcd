"""The quantiser's arithmetic step by step in numpy (fp32, the kernel's order) against the definition, for every bf16
value under every scale and for a reciprocal that is right or one ulp off: the kernel takes the hardware's, which
promises no more.  The clamp's limit is read from the kernel's source.  (No GPU.)"""

import os
import re

import numpy as np
import pytest

from oracle import cache_q4

CU = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_sharded_mla_gb300", "csrc",
                  "dcp_cache_q4.cu")
F = np.float32
BF16 = (np.arange(0, 0x7F80, dtype=np.uint32) << 16).view(F)     # every finite magnitude


def limit():
    text = open(CU).read()
    named = re.search(r"constexpr float kClampFrom = ([0-9.]+)f;", text)
    used = re.search(r"clamp = !\(top \* inv < ([0-9.]+f|kClampFrom)\)", text).group(1)
    return F(named.group(1) if used == "kClampFrom" else used[:-1])


def codes(x, s, inv, clamp):
    """codes8 of the kernel: snap to a multiple of 2^-11, then to a whole number that the low bits hold as code + 8."""
    snap, whole = F(6144.0), F(12582912.0 + 8.0)
    x = np.where(clamp, np.clip(x, F(-7) * s, F(7) * s), x)
    # the fused multiply-add: the product of two 24-bit numbers is exact in 64 bits, and so is the sum here
    a = (x.astype(np.float64) * inv.astype(np.float64) + float(snap)).astype(F)
    return ((a + (whole - snap)).view(np.uint32) & 0xFFFF).astype(np.int64) - 8


@pytest.mark.parametrize("off", [-1, 0, 1])
def test_codes_with_a_reciprocal_one_ulp_off(off):
    # the groups' scales by their largest magnitude, as the definition has them
    want = np.minimum(BF16.astype(np.float64) / 7, 448)
    up = np.clip(np.searchsorted(cache_q4.E4M3, want), 1, 126)
    a, b = want - cache_q4.E4M3[up - 1], cache_q4.E4M3[up] - want
    scale = np.where((a < b) | ((a == b) & ((up - 1) % 2 == 0)), up - 1, up)
    lim = limit()
    for e in range(1, 127):
        s = F(cache_q4.E4M3[e])
        inv = F(1) / s
        inv = np.nextafter(inv, F(np.inf) if off > 0 else F(0)) if off else inv
        tops = BF16[scale == e]
        assert len(tops)
        # every value of a group whose top does not clamp it, and the tops themselves
        clamp = ~(tops * inv < lim)
        x = BF16[BF16 <= tops.max()]
        for v, c in ((tops, clamp), (-tops, clamp), (x, np.full(len(x), bool(clamp.any()))),
                     (x[x <= tops[~clamp].max()] if not clamp.all() else x[:0], False)):
            true = np.clip(np.round(v.astype(np.float64) / float(s)), -7, 7)
            got = codes(v, s, np.broadcast_to(inv, v.shape), np.broadcast_to(c, v.shape))
            assert np.array_equal(got, true), (e, float(s), off)


@pytest.mark.gpu
def test_groups_at_the_clamp_bit_for_bit():
    """Tops of 7.5 times a scale (the smallest six and the largest), and the bf16 values beside them, of either sign."""
    import torch

    import context_sharded_mla_gb300 as dcp
    from test_gpu_q4 import store_rows
    tops = [7.5 * k / 512 for k in range(1, 8)] + [7.5 * 448]
    near = torch.tensor(tops).to(torch.bfloat16).view(torch.int16)
    tops = torch.cat([near - 1, near, near + 1]).view(torch.bfloat16).float()
    T = 2 * len(tops)
    g = torch.Generator().manual_seed(1)
    rows = torch.zeros(T, 36, 16)
    for t in range(T):
        top = float(tops[t // 2]) * (-1) ** t
        rows[t] = (torch.rand(36, 16, generator=g) * 2 - 1) * abs(top)
        rows[t, :, 3], rows[t, :, 9] = top, -top * 5 / 6
    rows = rows.flatten(1).to(torch.bfloat16)
    pages = -(-T // 8)
    arena = torch.zeros(1, pages * 8, 416, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_append_q4(dcp.Layout(1, 1, 8), 0, 1, rows.cuda(), torch.arange(T, device="cuda"),
                         torch.zeros(T, dtype=torch.int32, device="cuda"),
                         torch.arange(pages, dtype=torch.int32, device="cuda")[None], pages, arena, pages, status)
    assert int(status.item()) == 0
    assert np.array_equal(arena[0, :T].cpu().numpy(), store_rows(rows))
