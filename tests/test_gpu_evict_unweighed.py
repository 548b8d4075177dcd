"""Eviction of rows that have no weight yet: appended since the last weights were taken, or of a request that was shorter
than its queries.  They stay before any row that has a weight, and start from 0 when weights are taken next."""

import numpy as np
import pytest
import torch

import workloads
from oracle import evict, layout as olayout

from harness import to_f64
from test_gpu_evict_steps import Run

pytestmark = pytest.mark.gpu


class Tracked(Run):
    """A run with the weights that the definition gives, by position (+inf: none yet)."""

    def __init__(self, cache, **kw):
        super().__init__(cache, **kw)
        self.lens, self.w = [0] * self.B, [np.zeros(0) for _ in range(self.B)]

    def at(self, S):
        p = np.arange(S)
        return olayout.owner(p, self.N, self.I), olayout.local_row(p, self.N, self.I)

    def append(self, lens):
        """Rows in, no weights taken."""
        self.draw()
        self.new.copy_(torch.tensor(lens))
        pos, req = self.tables.update(self.new)
        self.dec.append_normed(self.kv, pos, req, self.tables.block_table, gamma=self.gamma, inv_freq=self.freq,
                               rope_pos=torch.where(pos >= 0, pos + self.shift[req.clamp(min=0).long()], -1))
        self.lens = lens
        self.w = [np.concatenate([w, np.full(S - len(w), np.inf)]) for w, S in zip(self.w, lens)]

    def weigh(self):
        self.q.copy_(torch.randn(self.q.shape, generator=self.g).to(torch.bfloat16))
        self.dec.decode(self.q, self.tables.block_table, self.tables.seq_lens)
        self.dec.weigh(self.q, self.tables.block_table, self.tables.seq_lens)
        got = to_f64(self.dec.weights)
        for b, S in enumerate(self.lens):
            w, _ = evict.key_weights(to_f64(self.q[b]), self.rows(b, S), S, workloads.SCALE, to_f64(self.dec.lse[b]), 0)
            want = np.where(np.isinf(self.w[b]), 0.0, self.w[b]) + w
            own, row = self.at(S)
            assert np.allclose(got[own, b, row], want, rtol=1e-4, atol=1e-30), b
            self.w[b] = got[own, b, row]

    def evict(self, new, sinks, recent):
        before = [self.rows(b, S) for b, S in enumerate(self.lens)]
        lens = self.lens
        self.new.copy_(torch.tensor(new))
        self.shrink(sinks, recent)
        for b, (S, m) in enumerate(zip(lens, new)):
            own, row = self.at(S)
            after, w = self.rows(b, m), np.zeros(m)
            for s in range(self.N):
                mine = np.zeros(len(row), np.float32)
                mine[row[own == s]] = self.w[b][own == s]
                kept = evict.select(mine, s, S, m, self.N, self.I, sinks, recent)
                assert self.dec.kept[s, b, :len(kept)].tolist() == kept, (b, s)
                for i, k in enumerate(kept):
                    to, frm = olayout.global_pos(s, i, self.N, self.I), olayout.global_pos(s, k, self.N, self.I)
                    assert np.array_equal(after[to], before[b][frm])
                    w[to] = self.w[b][frm]
            self.w[b] = w
        self.lens = new


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_rows_appended_since_the_last_weights(cache):
    r = Tracked(cache, seed=5)
    r.append([200, 33, 129])
    r.weigh()
    r.evict([120, 33, 60], 4, 8)                # behind the new lengths lie the weights of rows that went
    r.append([127, 38, 61])
    r.evict([118, 30, 59], 4, 2)                # light rows go, not those that nothing has weighed
    r.append([121, 31, 64])
    r.evict([117, 28, 58], 2, 0)                # twice without weights in between
    r.weigh()
    r.append([119, 30, 70])
    r.evict([119, 30, 70], 0, 0)                # nothing goes; the new rows are still without a weight
    r.append([130, 31, 71])
    r.weigh()
    r.evict([60, 20, 5], 4, 8)
    assert r.dec.status_bits() == 0 and r.tables.status_bits() == 0


def test_a_cache_that_was_never_weighed():
    r = Tracked("bf16", seed=6)
    r.dec.weights.copy_(torch.rand(r.dec.weights.shape, generator=r.g))     # what another request left
    r.append([90, 40, 11])
    r.evict([50, 39, 11], 3, 20)
    r.weigh()


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_a_request_shorter_than_its_queries_gets_no_weights(cache):
    import context_sharded_mla_gb300 as dcp
    from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
    lay, B, H = dcp.Layout(2, 1, 16), 2, 8
    d = ShardedMlaDecoder(lay, B, 2, H, 32, 8, workloads.SCALE, out_dtype=torch.float32, cache=cache, evict=True)
    tables = BlockTables(lay, B, 32, 8, max_tokens=128)
    d.weights.fill_(7.0)                        # what the slots' last requests left
    g = torch.Generator().manual_seed(4)
    for lens, status in (([1, 50], 16), ([3, 52], 0)):
        pos, req = tables.update(torch.tensor(lens, device="cuda"))
        d.append(torch.randn(128, 576, generator=g).to(torch.bfloat16).cuda(), pos, req, tables.block_table)
        q = torch.randn(B, 2, H, 576, generator=g).to(torch.bfloat16).cuda()
        d.decode(q, tables.block_table, tables.seq_lens)
        d.status.zero_()
        d.weigh(q, tables.block_table, tables.seq_lens)
        assert d.status_bits() == status
        if status:
            assert torch.all(d.weights[:, 0] == 7.0) and d.weighed.tolist() == [0, 50]
    assert d.weighed.tolist() == lens
    total = d.weights[0, 0, :2].sum() + d.weights[1, 0, :1].sum()
    assert abs(float(total) - 2 * H) < 1e-3     # the weights of 2 H query rows; 7 for each old row would show
    assert torch.all(d.weights[0, 0, 2:] == 7.0) and torch.all(d.weights[1, 0, 1:] == 7.0)


@pytest.mark.parametrize("N,I,begin,end", [(1, 1, 0, 1), (4, 2, 1, 3), (3, 8, 0, 3)])
@pytest.mark.parametrize("width", [1, 50, 9000])
def test_marked_rows(N, I, begin, end, width):
    import context_sharded_mla_gb300 as dcp
    lens = [0, 1, 40, width * N, width * N + 17, -3, 3 * width, 10 ** 12]
    first = [0, 0, 39, 5, width * N - 3, -4, 3 * width, -1]
    w = torch.rand(end - begin, len(lens), width, generator=torch.Generator().manual_seed(1))
    want = w.clone()
    for r in range(begin, end):
        for b, (f, S) in enumerate(zip(first, lens)):
            a, e = (min(width, int(olayout.count(r, max(0, x), N, I))) for x in (f, S))
            want[r - begin, b, a:e] = float("inf")
    got, side = w.cuda(), torch.cuda.Stream()
    args = (torch.tensor(first, device="cuda"), torch.tensor(lens, device="cuda"))
    torch.cuda.synchronize()
    dcp.dcp_key_weights_mark(dcp.Layout(N, I, 8), begin, end, *args, got, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("lens,q_len,H", [([700, 90], 1, 24), ([300], 33, 64)])   # the second shares its tiles
def test_marked_rows_start_from_nothing(q4, lens, q_len, H):
    from test_gpu_weigh import Case
    c = Case(lens, q_len, H, 2, 1, 16, q4=q4)
    before = c.fresh()
    marked = before.clone()
    marked[:, :, 3:20] = float("inf")
    zeroed = before.clone()
    zeroed[:, :, 3:20] = 0.0
    old = torch.tensor([S - q_len for S in lens], device="cuda")
    for decay in (1.0, 0.5, 0.0):
        w = c.run(marked.clone(), old, decay)
        assert torch.equal(w, c.run(zeroed.clone(), old, decay)) and not torch.isinf(w).any()


def test_refused_requests_keep_their_rows_and_weights():
    r = Tracked("bf16", seed=8)
    r.append([90, 40, 61])
    r.weigh()
    r.append([91, 42, 63])
    before, w = [r.rows(b, S) for b, S in enumerate(r.lens)], r.dec.weights.clone()
    r.dec.evict(r.tables.block_table, r.tables.seq_lens, torch.tensor([-1, 43, 63], device="cuda"), 2, 3)
    assert r.dec.status_bits() == 16 and r.dec.weighed.tolist() == [91, 42, 63]
    for b, (S, had) in enumerate(zip(r.lens, [90, 40, 61])):
        assert np.array_equal(r.rows(b, S), before[b])
        own, row = (torch.from_numpy(x).cuda() for x in r.at(S))
        assert torch.equal(r.dec.weights[own[:had], b, row[:had]], w[own[:had], b, row[:had]])
        assert torch.isinf(r.dec.weights[own[had:], b, row[had:]]).all()
    r.dec.status.zero_()
    r.weigh()                                   # and go on from there
    assert r.dec.status_bits() == 0
