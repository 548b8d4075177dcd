"""A serving run with eviction on both caches: rows normed and rotated into the shards, decode, weights, eviction, tables
that shrink, and decode over what is left; eagerly and captured."""

import numpy as np
import pytest
import torch

import workloads
from oracle import attention, cache_q4, evict, layout as olayout

from harness import assert_close_o, assert_close_lse, to_f64

pytestmark = pytest.mark.gpu

FREQ = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float()


class Run:
    def __init__(self, cache, B=3, H=24, N=4, I=2, P=16, pool=64, max_pages=16, seed=1):
        import context_sharded_mla_gb300 as dcp
        from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
        self.dcp, self.B, self.H, self.N, self.I, self.P, self.cache = dcp, B, H, N, I, P, cache
        lay = dcp.Layout(N, I, P)
        self.dec = ShardedMlaDecoder(lay, B, 1, H, pool, max_pages, workloads.SCALE, out_dtype=torch.float32, cache=cache,
                                     evict=True)
        self.tables = BlockTables(lay, B, pool, max_pages, max_tokens=1024)
        g = torch.Generator().manual_seed(seed)
        self.gamma = (1 + 0.2 * torch.randn(512, generator=g)).cuda()
        self.gamma_q = (1 + 0.2 * torch.randn(192, generator=g)).to(torch.bfloat16).cuda()
        self.w_kc = (torch.randn(H, 128, 512, generator=g) / 12).to(torch.bfloat16).cuda()
        self.freq = FREQ.cuda()
        self.kv = torch.zeros(1024, 576, dtype=torch.bfloat16, device="cuda")
        self.raw_q = torch.zeros(B, H, 192, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(B, 1, H, 576, dtype=torch.bfloat16, device="cuda")
        self.new = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.text = torch.zeros(B, dtype=torch.int64, device="cuda")    # places in the text, cache positions apart
        self.shift = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.g = g

    def draw(self):
        self.kv.copy_(torch.randn(1024, 576, generator=self.g).to(torch.bfloat16))
        self.raw_q.copy_((2 * torch.randn(self.B, self.H, 192, generator=self.g)).to(torch.bfloat16))

    def grow(self):
        """To the lengths in self.new: tables, rows in, queries, decode, weights."""
        pos, req = self.tables.update(self.new)
        rope = torch.where(pos >= 0, pos + self.shift[req.clamp(min=0).long()], -1)
        self.dec.append_normed(self.kv, pos, req, self.tables.block_table, gamma=self.gamma, inv_freq=self.freq, rope_pos=rope)
        self.dcp.dcp_q_norm_rope(self.raw_q, self.new + self.shift - 1, self.raw_q, gamma=self.gamma_q, inv_freq=self.freq)
        self.dcp.dcp_absorb_q(self.raw_q[..., :128].unsqueeze(1), self.raw_q[..., 128:].unsqueeze(1), self.w_kc, self.q)
        self.dec.decode(self.q, self.tables.block_table, self.tables.seq_lens)
        self.dec.weigh(self.q, self.tables.block_table, self.tables.seq_lens)

    def shrink(self, sinks, recent):
        self.dec.evict(self.tables.block_table, self.tables.seq_lens, self.new, sinks, recent)
        self.shift += self.tables.seq_lens - self.new
        self.tables.update(self.new)

    def rows(self, b, S):
        """Request b's cached values by position, as the host finds them."""
        arena, bt = self.dec.arena.cpu(), self.tables.block_table.cpu().numpy()
        p = np.arange(S)
        own, row = olayout.owner(p, self.N, self.I), olayout.local_row(p, self.N, self.I)
        x = arena[torch.from_numpy(own), torch.from_numpy(bt[b, row // self.P].astype(np.int64) * self.P + row % self.P)]
        return cache_q4.unpack(x.numpy()) if self.cache == "q4" else to_f64(x)

    def check_decode(self, lens):
        for b, S in enumerate(lens):
            o, lse, _, _ = attention.sharded_attention(to_f64(self.q[b]), self.rows(b, S), S, self.N, self.I, workloads.SCALE, 0)
            assert_close_o(to_f64(self.dec.o[b]), o, f"o of request {b}")
            assert_close_lse(to_f64(self.dec.lse[b]), lse, f"lse of request {b}")


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_a_serving_run_with_evictions(cache):
    r = Run(cache)
    lens = [200, 33, 129]
    weights = [np.zeros(0) for _ in lens]        # by position, as the oracle has them
    for step in range(6):
        r.draw()
        lens = [x + (1 if step else 0) for x in lens]
        r.new.copy_(torch.tensor(lens))
        r.grow()
        r.check_decode(lens)
        got = to_f64(r.dec.weights)
        for b, S in enumerate(lens):
            rows = r.rows(b, S)
            w, _ = evict.key_weights(to_f64(r.q[b]), rows, S, workloads.SCALE, to_f64(r.dec.lse[b]), 0)
            weights[b] = np.concatenate([weights[b], np.zeros(S - len(weights[b]))]) + w
            p = np.arange(S)
            own, row = olayout.owner(p, r.N, r.I), olayout.local_row(p, r.N, r.I)
            assert np.allclose(got[own, b, row], weights[b], rtol=1e-4, atol=1e-30)
        if step in (2, 4):
            before = [r.rows(b, S) for b, S in enumerate(lens)]
            free = int(r.tables.free_state[1])
            new = [120, 33, 20] if step == 2 else [60, 30, 20]
            new = [min(a, b) for a, b in zip(new, lens)]
            r.new.copy_(torch.tensor(new))
            r.shrink(4, 8)
            assert int(r.tables.free_state[1]) >= free
            for b, (S, m) in enumerate(zip(lens, new)):
                after, w = r.rows(b, m), np.zeros(m)
                for s in range(r.N):
                    mine = to_f64(torch.from_numpy(got[s, b]).float()).astype(np.float32)
                    kept = evict.select(mine, s, S, m, r.N, r.I, 4, 8)
                    assert r.dec.kept[s, b, :len(kept)].tolist() == kept
                    for i, k in enumerate(kept):
                        to, frm = olayout.global_pos(s, i, r.N, r.I), olayout.global_pos(s, k, r.N, r.I)
                        assert np.array_equal(after[to], before[b][frm])
                        w[to] = weights[b][frm]
                weights[b] = w
            lens = new
    assert r.dec.status_bits() == 0 and r.tables.status_bits() == 0


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_captured_steps_and_evictions(cache):
    """One graph for a step that grows, one for an eviction: replayed, they give what the calls give, bit for bit."""
    plan = [([150, 40, 90], False), ([151, 41, 91], False), ([100, 41, 30], True), ([101, 42, 31], False), ([50, 42, 31], True),
            ([51, 43, 32], False)]
    eager, held = Run(cache, seed=7), Run(cache, seed=7)
    # graphs of a run that is thrown away afterwards: its buffers go back to where they began
    graphs = {}
    start = {k: v.clone() for k, v in held.dec.__dict__.items() if isinstance(v, torch.Tensor)}
    start_t = {k: v.clone() for k, v in held.tables.__dict__.items() if isinstance(v, torch.Tensor)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held.new.fill_(5)
        held.grow()
        held.new.fill_(3)
        held.shrink(1, 1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for name, fn in (("grow", held.grow), ("shrink", lambda: held.shrink(4, 8))):
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            fn()
    for src, obj in ((start, held.dec), (start_t, held.tables)):
        for k, v in src.items():
            getattr(obj, k).copy_(v)
    held.shift.zero_()
    for lens, evicts in plan:
        for r in (eager, held):
            r.g.manual_seed(sum(lens))
            r.draw()
            r.new.copy_(torch.tensor(lens))
        if evicts:
            eager.shrink(4, 8)
            graphs["shrink"].replay()
        else:
            eager.grow()
            graphs["grow"].replay()
        torch.cuda.synchronize()
        for k in ("o", "lse", "weighed"):
            assert torch.equal(getattr(eager.dec, k), getattr(held.dec, k)), (lens, k)
        assert torch.equal(eager.tables.block_table, held.tables.block_table)
        for b, S in enumerate(lens):
            assert np.array_equal(eager.rows(b, S), held.rows(b, S))
    assert held.dec.status_bits() == 0 and held.tables.status_bits() == 0


def test_weights_and_evictions_of_a_ranks_shards():
    """Two decoders that hold half of the shards each, given the whole query and merged lse, do what one with all of them does."""
    whole = Run("bf16", seed=3)
    whole.draw()
    lens = [130, 77, 64]
    whole.new.copy_(torch.tensor(lens))
    whole.grow()
    before = whole.dec.arena.clone()
    from context_sharded_mla_gb300.step import ShardedMlaDecoder
    halves = []
    for a, e in ((0, 2), (2, 4)):
        d = ShardedMlaDecoder(whole.dec.layout, 3, 1, whole.H, whole.dec.pool_pages, whole.dec.max_pages, workloads.SCALE,
                              shard_begin=a, shard_end=e, evict=True)
        d.arena.copy_(before[a:e])
        d.lse.copy_(whole.dec.lse)
        d.weigh(whole.q, whole.tables.block_table, whole.tables.seq_lens)
        assert torch.equal(d.weights, whole.dec.weights[a:e])
        halves.append(d)
    new = torch.tensor([70, 70, 3], device="cuda")
    whole.dec.evict(whole.tables.block_table, whole.tables.seq_lens, new, 2, 5)
    for d, (a, e) in zip(halves, ((0, 2), (2, 4))):
        d.evict(whole.tables.block_table, whole.tables.seq_lens, new, 2, 5)
        assert torch.equal(d.arena, whole.dec.arena[a:e]) and torch.equal(d.weights, whole.dec.weights[a:e])
        assert d.status_bits() == 0


def test_two_threads_at_once():
    """Weights, selection and move from two host threads, a stream each, give what they give one after the other."""
    import threading
    runs = [Run("bf16", seed=11), Run("q4", seed=12)]
    want = [Run("bf16", seed=11), Run("q4", seed=12)]

    def go(r):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for lens, evicts in (([180, 60, 40], False), ([181, 61, 41], False), ([90, 61, 11], True), ([91, 62, 12], False)):
                r.new.copy_(torch.tensor(lens))
                r.shrink(2, 6) if evicts else r.grow()
        stream.synchronize()

    for r in runs + want:
        r.draw()
    torch.cuda.synchronize()
    for r in want:
        go(r)
    threads = [threading.Thread(target=go, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r, w in zip(runs, want):
        assert torch.equal(r.dec.o, w.dec.o) and torch.equal(r.dec.weighed, w.dec.weighed)
        for b, S in enumerate([91, 62, 12]):
            assert np.array_equal(r.rows(b, S), w.rows(b, S))
        assert r.dec.status_bits() == 0
