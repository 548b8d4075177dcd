"""The rotation's angles, sines and cosines, where a rotated value is small beside the pair it comes from: rounding to bf16
hides their errors elsewhere.

Bound (u = 2^-24) of a cos t - b sin t.  The angle: a step of 2^-64 turns off by 1.5 * 2^-53 of itself and 2^-65, times
the position (here below 2^20: 2^-32 rad and less), cut to 2^-32 turns and rounded to f32, half a last place of half a turn
(2^-25 of pi): below 2^-23.  Its sine and cosine one last place, at most u.  One product and one fused product and sum:
u |b| and u of the result.  In all (2^-23 + 2 u) (|a| + |b|) = 2^-22 (|a| + |b|), u of the result, and half a step of bf16,
2^-8 of it."""

import numpy as np
import pytest
import torch

from oracle import norm_rope

from harness import to_f64
from test_gpu_norm_rope import FREQ, run_append
from test_gpu_q4 import make_tables

pytestmark = pytest.mark.gpu


def check(got, x, pos, halves):
    want = norm_rope.rotate(x, pos, FREQ.double().numpy(), halves)
    i = np.arange(64)
    size = np.abs(x) + np.abs(x[..., (i + 32) % 64 if halves else i ^ 1])
    slack = 2.0 ** -22 * size + 2.0 ** -24 * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= slack + 2.0 ** -8 * (np.abs(want) + slack)), float(((err - 2.0 ** -8 * np.abs(want)) / size).max() * 2 ** 22)


@pytest.mark.parametrize("halves", [False, True])
def test_small_values_of_large_pairs(halves):
    import context_sharded_mla_gb300 as dcp
    g = torch.Generator().manual_seed(17)
    T, H = 60000, 2
    q = torch.randn(T, H, 192, generator=g)
    q[:, 1, 128:] *= torch.where(torch.rand(T, 64, generator=g) < 0.5, 2.0 ** -9, 1.0)   # angles near the axes too
    q = q.to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    out = torch.empty_like(q).cuda()
    dcp.dcp_q_norm_rope(q.cuda(), pos.cuda(), out, inv_freq=FREQ.cuda(), rope_style=int(halves))
    check(to_f64(out)[..., 128:], to_f64(q)[..., 128:], pos.numpy(), halves)


@pytest.mark.parametrize("halves", [False, True])
def test_small_values_of_large_pairs_in_the_cache(halves):
    g = torch.Generator().manual_seed(18)
    T, P = 60000, 64
    x = torch.randn(T, 576, generator=g).to(torch.bfloat16)
    bt, pool = make_tables([T], 1, P, 0, 3)
    pos, rope = torch.arange(T), torch.randint(0, 1 << 20, (T,), generator=g)
    arena, status = run_append(False, x.cuda(), pos.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"),
                               torch.from_numpy(bt).cuda(), pool, 1, 1, P, 0, 1, inv_freq=FREQ.cuda(), rope_style=int(halves),
                               rope_pos=rope.cuda())
    assert status == 0
    rows = arena[0, torch.from_numpy(bt[0, np.arange(T) // P].astype(np.int64) * P + np.arange(T) % P).cuda()]
    check(to_f64(rows)[:, 512:], to_f64(x)[:, 512:], rope.numpy(), halves)
