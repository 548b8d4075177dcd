"""Weights under the library's own lse: how far a query row's sum is from one, and how much of that grows with the score.

The mean over 512 query rows of the sum's distance from one, in u = 2^-24, against the mean score s that carries the
weights (natural logarithms).

Roundings.  The decode's x = s c - m and the weights' x = s c - lse2 are one fused step each (u |x|, |x| small where the
weights are), exp2 is off by 4 u either way, a row's sums are of positive terms; lse2 itself is rounded once or twice
(u s each, independent from row to row: over 512 rows four deviations are 0.15 u s).  Together below u s / 4 + 8 u.

Scores of two terms that f32 holds exactly leave nothing for the tensor core to cut off: what is left is the correction
of the scores' scale, 8 u (its product rounded to f32: half a unit more) on a bf16 cache, none on a 4-bit one.

Dense scores: a step of a sum cuts half a last place of the sum so far on average, u of it at most.  A sum that grows evenly
over 36 steps loses 36 u / 2 = 18 u of the score at most, the decode's two halves of 18 steps each half of that: what the
weights' scores are lower lies in [0, 9 u] of a bf16 score and is corrected by 8 u, and in as much of a 4-bit one, whose
values have half the bits and lose less than half: 8 u s and 4.5 u s."""

import math

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bias(cache, q, kv):
    """(mean distance of a query row's sum from one, mean score) of q [B, 1, H, 576] over kv [B, S, 576]."""
    import context_sharded_mla_gb300 as dcp
    from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
    B, _, H, _ = q.shape
    S = kv.shape[1]
    lay = dcp.Layout(2, 1, 16)
    pages = -(-S // 32)
    d = ShardedMlaDecoder(lay, B, 1, H, B * pages, pages, workloads.SCALE, lse_base=dcp.DCP_LSE_BASE_2, cache=cache, evict=True)
    tables = BlockTables(lay, B, B * pages, pages, max_tokens=B * S)
    pos, req = tables.update(torch.full((B,), S, device="cuda"))
    d.append(kv.reshape(-1, 576).cuda(), pos, req, tables.block_table)
    _, lse = d.decode(q.cuda(), tables.block_table, tables.seq_lens)
    w = d.weigh(q.cuda(), tables.block_table, tables.seq_lens)
    assert d.status_bits() == 0 and tables.status_bits() == 0
    return float(w.double().sum()) / (B * H) - 1, float(lse.double().mean()) * math.log(2)


@pytest.mark.parametrize("cache,factor", [("bf16", 8.5), ("q4", 0)])
def test_scores_of_two_exact_terms(cache, factor):
    g = torch.Generator().manual_seed(9)
    B, H, S = 4, 128, 300
    q, kv = torch.zeros(B, 1, H, 576), torch.zeros(B, S, 576)
    for d in (520, 571):                                   # position dims: bf16 in either cache
        q[..., d] = torch.randint(8, 40, (B, 1, H), generator=g)
        kv[..., d] = torch.randint(1, 24, (B, S), generator=g)
    off, s = bias(cache, q.to(torch.bfloat16), kv.to(torch.bfloat16))
    assert 40 < s < 200
    assert abs(off) <= (factor + 0.25) * U * s + 8 * U, off / U / s


@pytest.mark.parametrize("cache,factor", [("bf16", 8.5), ("q4", 4.5)])
@pytest.mark.parametrize("size", [1.0, 4.0, 16.0])
def test_dense_scores(cache, factor, size):
    g = torch.Generator().manual_seed(10)
    q = (size * torch.randn(4, 1, 128, 576, generator=g)).to(torch.bfloat16)
    kv = torch.randn(4, 700, 576, generator=g).to(torch.bfloat16)
    off, s = bias(cache, q, kv)
    assert abs(off) <= (factor + 0.25) * U * s + 8 * U, off / U / s
