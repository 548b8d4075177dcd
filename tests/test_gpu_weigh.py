"""Attention weight of cached rows on the GPU (both caches), against fp64 over what the cache holds.

Bounds, from the roundings (u = 2^-24).  A term is 2^x, x = s log2 e - lse2.  The score is a dot product of 576 exact
bf16 products added in fp32, at most 2 u each step: |ds| <= 576 * 2 u * scale * sum_d |q_d k_d|.  x has the rounding of
the scale (u |s|), of lse's base change (2 u |lse|) and of one fma (u |x|), in all below 2^-21 (1 + |s| + |lse|), exp2 is
off by 2^-22.  Terms are positive, so R of them add at most R u of their sum, the old weight two more roundings.  A term
below 2^-126 may be 0."""

import numpy as np
import pytest
import torch

import workloads
from oracle import cache_q4, evict, layout as olayout

from harness import to_f64
from test_gpu_q4 import make_tables, random_rows, store_rows

pytestmark = pytest.mark.gpu

SCALE = workloads.SCALE
U = 2.0 ** -24


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def scores(q, kv):
    """q [q_len, H, 576] . kv [S, 576] -> [q_len, H, S]."""
    return (q.reshape(-1, 576) @ kv.T).reshape(*q.shape[:2], len(kv))


class Case:
    """Requests in a cache (rows that belong to nobody are NaN), their queries and merged lse."""

    def __init__(self, lens, q_len, H, N, I, P, begin=0, end=None, base=0, q4=False, seed=1, spare=2, extra=3):
        dcp = _dcp()
        self.lens, self.q_len, self.H, self.N, self.I, self.P, self.base, self.q4 = lens, q_len, H, N, I, P, base, q4
        self.begin, self.end = begin, N if end is None else end
        self.layout = dcp.Layout(N, I, P)
        bt, self.pool = make_tables(lens, N, P, spare, seed)
        self.bt_host, self.bt = bt, torch.from_numpy(bt).cuda()
        n, B = self.end - self.begin, len(lens)
        g = torch.Generator().manual_seed(seed)
        self.kv = [random_rows(max(1, S), seed + 10 + b)[:S] for b, S in enumerate(lens)]
        if q4:
            arena = np.full((n, self.pool * P, 416), 255, np.uint8)
            rows = [store_rows(x) if len(x) else None for x in self.kv]
            self.values = [cache_q4.unpack(x) if x is not None else np.zeros((0, 576)) for x in rows]
        else:
            arena = np.full((n, self.pool * P, 576), 0x7FC0, np.uint16)
            rows = [x.view(torch.int16).numpy().view(np.uint16) for x in self.kv]
            self.values = [to_f64(x) for x in self.kv]
        for b, S in enumerate(lens):
            p = np.arange(S)
            own, row = olayout.owner(p, N, I), olayout.local_row(p, N, I)
            keep = (own >= self.begin) & (own < self.end)
            arena[own[keep] - self.begin, bt[b, row[keep] // P] * P + row[keep] % P] = rows[b][keep] if S else 0
        self.arena = torch.from_numpy(arena if q4 else arena.view(np.int16)).cuda()
        if not q4:
            self.arena = self.arena.view(torch.bfloat16)
        self.q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16)
        self.lse = torch.zeros(B, q_len, H)
        for b, S in enumerate(lens):
            if S < q_len:
                continue
            s = scores(to_f64(self.q[b]), self.values[b]) * SCALE
            s = np.where(np.arange(S) <= (S - q_len + np.arange(q_len))[:, None, None], s, -np.inf)
            m = s.max(-1)
            self.lse[b] = torch.from_numpy(m + np.log(np.exp(s - m[..., None]).sum(-1)))
        if base:
            self.lse = self.lse / np.log(2.0)
        self.lse = self.lse.float()
        self.wide = bt.shape[1] * P + extra
        self.seq_lens = torch.tensor(lens, dtype=torch.int64, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, weights, old_lens=None, decay=1.0, q=None, lse=None, stream=None, arena=None, bt=None, workspace=None):
        dcp = _dcp()
        fn = dcp.dcp_mla_key_weights_q4 if self.q4 else dcp.dcp_mla_key_weights
        fn(self.layout, self.begin, self.end, (self.q if q is None else q).cuda(), self.arena if arena is None else arena,
           self.pool, self.bt if bt is None else bt, self.bt.shape[1], self.seq_lens, SCALE, self.base,
           (self.lse if lse is None else lse).cuda(), weights, self.status, old_lens=old_lens, decay=decay, stream=stream,
           workspace=workspace)
        return weights

    def fresh(self, seed=9):
        g = torch.Generator().manual_seed(seed)
        return torch.rand(self.end - self.begin, len(self.lens), self.wide, generator=g).cuda()

    def check(self, got, before, old_lens, decay):
        got, before = to_f64(got), to_f64(before)
        worst = 0.0
        for b, S in enumerate(self.lens):
            want, size = evict.key_weights(to_f64(self.q[b]), self.values[b], S, SCALE, to_f64(self.lse[b]), self.base)
            dots = scores(np.abs(to_f64(self.q[b])), np.abs(self.values[b]))
            ds = 576 * 2 * U * SCALE * dots.max((0, 1))
            p = np.arange(S)
            own, row = olayout.owner(p, self.N, self.I), olayout.local_row(p, self.N, self.I)
            for r in range(self.begin, self.end):
                at = p[own == r]
                g, w0 = got[r - self.begin, b], before[r - self.begin, b]
                old = np.where(at < old_lens[b], decay * w0[row[at]], 0.0) if decay else np.zeros(len(at))
                ref = old + want[at]
                bound = (want[at] * (1.01 * ds[at] + (self.q_len * self.H + 4) * U) + 2.0 ** -21 * size[at] + 3 * U * np.abs(ref)
                         + self.q_len * self.H * 2.0 ** -126)
                err = np.abs(g[row[at]] - ref)
                assert np.all(err <= bound), (b, r, float((err / bound).max()))
                worst = max([worst, *(err / bound)])
                assert np.array_equal(g[len(at):], w0[len(at):])           # rows behind the last one
        return worst


CASES = [
    ([1024], 1, 16, 4, 1, 16, 0, 4, 0),
    ([1], 1, 1, 1, 1, 8, 0, 1, 0),
    ([1, 130, 4097, 63], 1, 96, 8, 1, 64, 0, 8, 1),
    ([300, 5, 1500], 4, 128, 4, 16, 64, 1, 3, 0),              # several groups of rows, half of the shards
    ([3, 700], 3, 5, 2, 8, 8, 0, 2, 1),
    ([513], 61, 7, 1, 1, 128, 0, 1, 0),                        # 427 rows, most of the keys behind a mask
    ([257, 800], 2, 128, 3, 2, 32, 0, 3, 0),                   # exactly 256 rows
    ([400], 1, 257, 2, 1, 64, 0, 2, 1),
    ([1400, 64], 64, 96, 2, 1, 64, 0, 2, 0),                   # a window of 64 queries
    ([2, 1, 3, 1, 7, 2, 9, 1] * 40, 1, 33, 16, 1, 8, 0, 16, 0),  # many short requests, empty shards
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("q4", [False, True])
def test_weights(case, q4):
    lens, q_len, H, N, I, P, begin, end, base = CASES[case]
    c = Case(lens, q_len, H, N, I, P, begin, end, base, q4)
    before = c.fresh()
    w = c.run(before.clone())                                  # no old_lens: every row starts from 0
    c.check(w, before, [0] * len(lens), 1.0)
    old_lens = [max(0, S - q_len - (b % 3)) for b, S in enumerate(lens)]
    old = torch.tensor(old_lens, dtype=torch.int64, device="cuda")
    for decay in (1.0, 0.75, 0.0):
        w = c.run(before.clone(), old, decay)
        c.check(w, before, old_lens, decay)
    again = c.run(before.clone(), old, 0.0)
    assert torch.equal(w, again)                               # equal calls, equal bits
    assert int(c.status.item()) == 0


SHARED = [  # few tiles for many query rows: pairs that share a tile, several of them inside one
    ([130], 33, 64, 1, 1, 16, 0, 1, 0),                        # one tile, more row groups than anything else
    ([3000, 12, 700], 11, 96, 2, 1, 64, 0, 2, 1),               # a request shorter than a tile between two
    ([9000], 11, 100, 4, 1, 64, 1, 3, 0),                      # five groups of rows; half of the shards
    ([16000, 16000], 9, 128, 1, 1, 128, 0, 1, 0),              # a tile and a part of one a run
    ([9700, 9700], 11, 100, 1, 1, 32, 0, 1, 0),                # a tile a run: none is shared
    ([64] * 9, 61, 40, 1, 1, 8, 0, 1, 0),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("q4", [False, True])
def test_shared_tiles(case, q4):
    """A workspace, its own and dirty, and none (tiles are not shared then); with weights to add to."""
    dcp = _dcp()
    c = Case(*SHARED[case], q4)
    before = c.fresh()
    old_lens = [max(0, S - c.q_len - b % 3) for b, S in enumerate(c.lens)]
    old = torch.tensor(old_lens, dtype=torch.int64, device="cuda")
    w = c.run(before.clone(), old, 0.5)
    c.check(w, before, old_lens, 0.5)
    size = (dcp.dcp_mla_key_weights_workspace_size_q4 if q4 else dcp.dcp_mla_key_weights_workspace_size)(c.q_len, c.H)
    dirty = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(w, c.run(before.clone(), old, 0.5, workspace=dirty))
    fn = dcp.load_library().dcp_mla_key_weights_q4 if q4 else dcp.load_library().dcp_mla_key_weights
    alone, q, lse = before.clone(), c.q.cuda(), c.lse.cuda()
    assert fn(c.layout, c.begin, c.end, q.data_ptr(), len(c.lens), c.q_len, c.H, c.arena.data_ptr(), c.pool, c.bt.data_ptr(),
              c.bt.stride(0), c.bt.shape[1], c.seq_lens.data_ptr(), SCALE, c.base, lse.data_ptr(), old.data_ptr(), 0.5,
              alone.data_ptr(), c.wide, None, 0, c.status.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    c.check(alone, before, old_lens, 0.5)
    assert int(c.status.item()) == 0


def test_shared_tiles_on_two_streams_and_in_graphs():
    """Scratch that the calls take for themselves: two calls at once on streams of their own, two graphs replayed together."""
    cases = [Case([2000, 300], 12, 96, 2, 1, 64, seed=s) for s in (1, 2)]
    qs, lses = [c.q.cuda() for c in cases], [c.lse.cuda() for c in cases]
    for c, k in zip(cases, range(2)):
        c.q, c.lse = qs[k], lses[k]
    want = [c.run(c.fresh()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [c.fresh() for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, s in zip(cases, got, streams):
            c.run(w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], [c.fresh() for c in cases]
    for c, w in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(w)
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(int(c.status.item()) == 0 for c in cases)


@pytest.mark.parametrize("q4", [False, True])
def test_weights_of_the_decodes_own_lse_sum_to_one(q4):
    """The lse of the partial decode and the merge of the same library: each query row's weights sum to one."""
    dcp = _dcp()
    lens, q_len, H, N, I, P = [900, 3001, 70], 2, 40, 4, 1, 16
    c = Case(lens, q_len, H, N, I, P, q4=q4)
    size = dcp.dcp_mla_decode_workspace_size_q4 if q4 else dcp.dcp_mla_decode_workspace_size
    part = dcp.dcp_mla_decode_partial_q4 if q4 else dcp.dcp_mla_decode_partial
    B = len(lens)
    arena = c.arena if q4 else torch.nan_to_num(c.arena, nan=0.0)    # the bf16 decode wants finite rows behind the last
    o = torch.empty(N, B, q_len, H, 512, device="cuda")
    z = torch.empty(N, B, q_len, H, device="cuda")
    ws = torch.empty(size(c.layout, 0, N, B, q_len, H), dtype=torch.uint8, device="cuda")
    part(c.layout, 0, N, c.q.cuda(), arena, c.pool, c.bt, c.bt.shape[1], c.seq_lens, SCALE, 0, o, z, ws, c.status)
    merged, lse = torch.empty(B * q_len * H, 512, device="cuda"), torch.empty(B, q_len, H, device="cuda")
    dcp.dcp_lse_merge(o.view(N, -1, 512), z.view(N, -1), 0, merged, lse.view(-1))
    w = c.run(torch.zeros(N, B, c.wide, device="cuda"), lse=lse)
    total = w.double().sum((0, 2)).cpu().numpy()
    assert np.all(np.abs(total - q_len * H) <= q_len * H * 2.0 ** -14)


@pytest.mark.parametrize("q4", [False, True])
def test_what_rows_and_queries_may_hold(q4):
    c = Case([200, 150], 2, 24, 2, 1, 16, q4=q4)
    before = c.fresh()
    clean = c.run(before.clone())
    arena = c.arena.clone()                                    # a NaN row: its own weight alone
    row = int(c.bt_host[0, 3] * 16 + 5)
    arena[1, row] = 255 if q4 else float("nan")
    w = c.run(before.clone(), arena=arena)
    bad = torch.isnan(w)
    assert bad[1, 0, 3 * 16 + 5] and int(bad.sum()) == 1
    assert torch.equal(w[~bad], clean[~bad])
    lse = c.lse.clone()                                        # a query row that saw nothing adds nothing
    lse[0, 1, 3] = float("-inf")
    w = c.run(before.clone(), lse=lse)
    assert torch.equal(w[:, 1], clean[:, 1]) and bool((w[:, 0, :100] < clean[:, 0, :100]).all())
    only = torch.full_like(c.lse, float("-inf"))
    assert not c.run(before.clone(), lse=only)[:, 0, :100].any()
    lse = c.lse.clone()                                        # a NaN lse: every row that query row sees
    lse[1, 0, 0] = float("nan")
    w = c.run(before.clone(), lse=lse)
    seen = torch.isnan(w)
    assert int(seen[:, 0].sum()) == 0 and int(seen[:, 1].sum()) == 149   # not the last token's own row
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("q4", [False, True])
def test_bad_pages_and_lengths(q4):
    c = Case([300, 3, 90], 4, 8, 2, 1, 8, q4=q4)
    before = c.fresh()
    w = c.run(before.clone())                                  # request 1 is shorter than its queries
    assert int(c.status.item()) == 16 and torch.equal(w[:, 1], before[:, 1])
    c.status.zero_()
    bt = c.bt.clone()
    bt[0, 2], bt[2, 0] = c.pool, -1
    w2 = c.run(before.clone(), bt=bt)
    assert int(c.status.item()) == 16 | 4
    same = torch.ones_like(w, dtype=torch.bool)
    same[:, 0, 16:24] = False
    same[:, 2, 0:8] = False
    assert torch.equal(w2[same], w[same]) and torch.equal(w2[~same], before[~same])
    c.status.zero_()
    c.seq_lens[2] = 10 ** 15                                   # longer than its table: as far as the table goes
    w3 = c.run(before.clone())
    assert int(c.status.item()) & 4
    assert torch.equal(w3[:, 0], w[:, 0])


@pytest.mark.parametrize("q4", [False, True])
def test_streams_and_graphs(q4):
    c = Case([700, 1300], 1, 96, 4, 1, 64, q4=q4)
    q, lse, old = c.q.cuda(), c.lse.cuda(), torch.tensor([650, 1300], device="cuda")
    before = c.fresh()
    want = c.run(before.clone(), old)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [before.clone() for _ in streams]
    torch.cuda.synchronize()
    for s, w in zip(streams, got):                             # two calls at once
        c.run(w, old, q=q, lse=lse, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(w, want) for w in got)
    held = before.clone()
    c.run(held, old, q=q, lse=lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.run(held, old, q=q, lse=lse)
    for _ in range(2):
        held.copy_(before)
        graph.replay()
        assert torch.equal(held, want)
    c.seq_lens[0] = 401                                        # the captured call reads the lengths
    held.copy_(before)
    graph.replay()
    c.lens = [401, 1300]
    # the keys of the shorter request are the first 401, seen by a query whose lse is still the longer one's
    c.values[0] = c.values[0][:401]
    c.check(held, before, [650, 1300], 1.0)


def test_rows_beyond_four_gigabytes():
    dcp = _dcp()
    P, pages = 64, 60000                                       # 60000 * 64 * 1152 bytes: 4.4 GB
    arena = torch.empty(1, pages * P, 576, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[pages - 1, 3, pages - 2, 58255]], dtype=torch.int32, device="cuda")
    x = random_rows(250, 3).cuda()
    for k in range(4):
        arena[0, int(ids[0, k]) * P:int(ids[0, k]) * P + len(x[64 * k:64 * k + 64])] = x[64 * k:64 * k + 64]
    q = torch.randn(1, 1, 20, 576, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    s = to_f64(q)[0, 0] @ to_f64(x).T * SCALE
    lse = np.log(np.exp(s).sum(-1))
    w = torch.zeros(1, 1, 256, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_mla_key_weights(dcp.Layout(1, 1, P), 0, 1, q.cuda(), arena, pages, ids, 4, torch.tensor([250], device="cuda"), SCALE, 0,
                            torch.from_numpy(lse).float().view(1, 1, 20).cuda(), w, status)
    want = np.exp(s - lse[:, None]).sum(0)
    assert int(status.item()) == 0
    assert np.all(np.abs(to_f64(w)[0, 0, :250] - want) <= 1e-4 * want)   # ds <= 576 * 2 u * 35, and the rest below 2^-16


def test_tensors_of_the_wrong_shape():
    c = Case([40], 1, 4, 1, 1, 8)
    good = c.fresh()
    for w in (good[0], good.repeat(1, 2, 1), good.double(), good.transpose(1, 2), good[..., :39]):
        with pytest.raises((ValueError, RuntimeError)):        # the last one is shorter than the block table: refused by the call
            c.run(w)
    with pytest.raises(ValueError):
        c.run(good, lse=c.lse[..., :3])
    with pytest.raises(ValueError):
        c.run(good, old_lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert int(c.status.item()) == 0
