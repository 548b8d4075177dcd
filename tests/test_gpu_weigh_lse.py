"""The lse that ShardedMlaDecoder.weigh takes: the merged one of all shards, of whatever queries are weighed."""

import numpy as np
import pytest
import torch

import workloads
from oracle import evict, layout as olayout

from harness import to_f64
from test_gpu_evict_steps import Run

pytestmark = pytest.mark.gpu


def halves_of(r, **kw):
    """Decoders with two of the run's four shards each, and its rows."""
    from context_sharded_mla_gb300.step import ShardedMlaDecoder
    out = []
    for a, e in ((0, 2), (2, 4)):
        d = ShardedMlaDecoder(r.dec.layout, r.B, 1, r.H, r.dec.pool_pages, r.dec.max_pages, workloads.SCALE, out_dtype=torch.float32,
                              cache=r.cache, shard_begin=a, shard_end=e, evict=True, **kw)
        d.arena.copy_(r.dec.arena[a:e])
        out.append(d)
    return out


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_some_of_the_shards_want_the_lse_of_all(cache):
    r = Run(cache, seed=21)
    r.draw()
    r.new.copy_(torch.tensor([130, 77, 64]))
    r.grow()
    args = (r.q, r.tables.block_table, r.tables.seq_lens)
    for d, at in zip(halves_of(r), (slice(0, 2), slice(2, 4))):
        d.decode(*args)                                  # d.lse: over its own shards alone
        with pytest.raises(ValueError, match="lse"):
            d.weigh(*args)
        assert not d.weights.any() and not d.weighed.any()
        d.weigh(*args, lse=r.dec.lse)
        assert torch.equal(d.weights, r.dec.weights[at]) and torch.equal(d.weighed, r.tables.seq_lens)
        assert d.status_bits() == 0


def test_no_weights_from_an_lse_that_nothing_wrote():
    r = Run("bf16", seed=22)
    r.draw()
    r.new.copy_(torch.tensor([130, 77, 64]))
    r.grow()
    for d in halves_of(r):
        d.weigh(r.q, r.tables.block_table, r.tables.seq_lens)
        for s in range(2):
            for b, S in enumerate([130, 77, 64]):
                n = int(olayout.count(d.shard_begin + s, S, r.N, r.I))
                assert torch.isnan(d.weights[s, b, :n]).all()


@pytest.mark.parametrize("cache", ["bf16", "q4"])
@pytest.mark.parametrize("q_len", [5, 60])               # 60 tokens of 24 heads share tiles, on more scratch than the decode's
def test_a_window_of_queries_on_a_decoder_of_single_tokens(cache, q_len):
    import context_sharded_mla_gb300 as dcp
    from oracle import attention
    r = Run(cache, seed=23)
    r.draw()
    lens = [200, 4, 129]                                 # the second is shorter than the window
    r.new.copy_(torch.tensor(lens))
    r.grow()
    had = r.dec.weighed.clone()
    before = to_f64(r.dec.weights)
    q = torch.randn(r.B, q_len, r.H, 576, generator=r.g).to(torch.bfloat16)
    lse = torch.zeros(r.B, q_len, r.H)
    for b, S in enumerate(lens):
        if S >= q_len:
            lse[b] = torch.from_numpy(np.asarray(attention.sharded_attention(to_f64(q[b]), r.rows(b, S), S, r.N, r.I, workloads.SCALE, 0)[1])
                                      .reshape(q_len, r.H))
    with pytest.raises(ValueError):
        r.dec.weigh(q.cuda(), r.tables.block_table, r.tables.seq_lens)      # self.lse is of one token
    r.dec.weigh(q.cuda(), r.tables.block_table, r.tables.seq_lens, decay=0.5, lse=lse.cuda())
    assert torch.equal(r.dec.weighed, had) and r.dec.status_bits() == 16
    got = to_f64(r.dec.weights)
    assert np.array_equal(got[:, 1], before[:, 1])
    for b in (0, 2):
        S = lens[b]
        w, _ = evict.key_weights(to_f64(q[b]), r.rows(b, S), S, workloads.SCALE, to_f64(lse[b]), 0)
        p = np.arange(S)
        own, row = olayout.owner(p, r.N, r.I), olayout.local_row(p, r.N, r.I)
        assert np.allclose(got[own, b, row], 0.5 * before[own, b, row] + w, rtol=1e-4, atol=1e-30)
