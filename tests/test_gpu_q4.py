"""The 4-bit latent cache on the GPU: append, relayout and read bit for bit, and the partial decode
against fp64 attention over the rows the cache holds.

Bounds of the partial decode, from its roundings (u = 2^-24, dot products of 576 exact bf16 products
summed in fp32 with at most 2u each):
  scores  |ds| <= 576 * 2u * scale * sum_d |q_d k_d|, its largest over the row's keys
  lse     ds + 2^-20 max(1, |lse|)          (exp2 and log2 approximations, fp32 sums of positive terms)
  o       (2^-8 + 2 ds + 2^-16) sum_p w_p |v_p|, the 2^-8 being the softmax weights' rounding to bf16;
          + 2^-8 |o| for bf16 partials
          + 2^-110 sum_p |v_p|: a weight is 2^(s - m) in fp32, which is 0 below 2^-126, for a reference m
          at most 8 off the row's largest score (in powers of two), over a sum of at least 2^-8
"""

import numpy as np
import pytest
import torch

import workloads
from oracle import attention, cache_q4, layout as olayout

from harness import to_f64

pytestmark = pytest.mark.gpu

SCALE = workloads.SCALE


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def make_tables(lens, N, P, spare, seed, max_pages=None):
    npages = [max(1, -(-int(x) // (N * P))) for x in lens]
    pool = sum(npages) + spare
    perm = np.random.default_rng(seed).permutation(pool).astype(np.int32)
    bt = np.full((len(lens), max_pages or max(npages)), -1, np.int32)
    off = 0
    for b, n in enumerate(npages):
        bt[b, :n] = perm[off:off + n]
        off += n
    return bt, pool


def store_rows(values):
    """416-byte rows the cache holds for bf16 rows [T, 576] (torch, CPU)."""
    v = to_f64(values)
    codes, scales = cache_q4.quantise(v[:, :512])
    return cache_q4.pack(codes, scales, values[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16))


def random_rows(T, seed, spread=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 576, generator=g)
    if spread:   # groups of every size e4m3 scales can have, zeros and ties among them
        x = x * torch.exp2(torch.randint(-14, 13, (T, 36), generator=g).float()).repeat_interleave(16, 1)
        x[::3, 16:32] = 0
        x[1::3, 32:48] = torch.randint(-14, 15, (len(x[1::3]), 16), generator=g).float() / 2
        x[1::3, 32] = 7.0
    return x.to(torch.bfloat16)


# ---------------------------------------------------------------- append / read / relayout
@pytest.mark.parametrize("N,I,P,begin,end", [(4, 1, 16, 0, 4), (8, 1, 64, 2, 5), (3, 8, 8, 0, 3), (1, 1, 8, 0, 1),
                                             (2, 16, 128, 1, 2)])
@pytest.mark.parametrize("spread", [False, True])
def test_append_and_read_bit_for_bit(N, I, P, begin, end, spread):
    dcp = _dcp()
    lens = [1, 37, 3 * N * P + 5]
    bt, pool = make_tables(lens, N, P, 2, 7)
    pos = np.concatenate([np.arange(n) for n in lens] + [[-1, -1]]).astype(np.int64)
    req = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[-1, -1]]).astype(np.int32)
    order = np.random.default_rng(1).permutation(len(pos))
    pos, req = pos[order], req[order]
    rows = random_rows(len(pos), 11, spread)
    want = store_rows(rows)
    n = end - begin
    fill = torch.randint(0, 256, (n, pool * P, 416), dtype=torch.uint8, generator=torch.Generator().manual_seed(3))
    arena = fill.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (torch.from_numpy(pos).cuda(), torch.from_numpy(req).cuda(), torch.from_numpy(bt).cuda(), bt.shape[1])
    dcp.dcp_kv_append_q4(dcp.Layout(N, I, P), begin, end, rows.cuda(), *args, arena, pool, status)
    ref = fill.numpy().copy()
    mine = np.zeros(len(pos), bool)
    for t, (p, b) in enumerate(zip(pos, req)):
        if p >= 0 and begin <= olayout.owner(p, N, I) < end:
            row = olayout.local_row(p, N, I)
            ref[olayout.owner(p, N, I) - begin, bt[b, row // P] * P + row % P] = want[t]
            mine[t] = True
    assert np.array_equal(arena.cpu().numpy(), ref)          # other rows, other shards' and padding untouched
    kv = torch.full((len(pos), 576), 5.0, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_read_q4(dcp.Layout(N, I, P), begin, end, arena, pool, *args, kv, status)
    got = to_f64(kv)
    assert np.array_equal(got[mine], cache_q4.unpack(want[mine]))
    assert np.all(got[~mine] == 5.0)
    assert int(status.item()) == 0


def test_append_of_infinities_and_nans():
    dcp = _dcp()
    rows = random_rows(3, 5)
    rows[0, 3], rows[1, 20], rows[1, 21] = float("inf"), float("-inf"), 4000.0
    rows[2, 40] = float("nan")
    rows[2, 530] = float("nan")
    arena = torch.zeros(1, 8, 416, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (torch.arange(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
            torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    lay = dcp.Layout(1, 1, 8)
    dcp.dcp_kv_append_q4(lay, 0, 1, rows.cuda(), *args, arena, 1, status)
    kv = torch.zeros(3, 576, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_read_q4(lay, 0, 1, arena, 1, *args, kv, status)
    got = to_f64(kv)
    assert got[0, 3] == 7 * 448 and got[1, 20] == -7 * 448 and got[1, 21] == 7 * 448
    assert np.all(np.isnan(got[2, 32:48])) and np.isnan(got[2, 530])
    assert np.isfinite(np.delete(got[2], list(range(32, 48)) + [530])).all() and np.isfinite(got[:2]).all()


@pytest.mark.parametrize("N,I,P,Ps,begin,end", [(8, 1, 64, 64, 0, 8), (4, 4, 16, 48, 1, 3), (1, 1, 8, 3, 0, 1)])
def test_relayout_bit_for_bit(N, I, P, Ps, begin, end):
    dcp = _dcp()
    lens = [5, 2 * N * P + 3, 70]
    bt, pool = make_tables(lens, N, P, 1, 9)
    sbt, spool = make_tables(lens, 1, Ps, 2, 10)
    src = random_rows(spool * Ps, 12, spread=True)
    want = store_rows(src)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int64)
    req = np.concatenate([np.full(n, b) for b, n in enumerate(lens)]).astype(np.int32)
    arena = torch.zeros(end - begin, pool * P, 416, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_relayout_q4(dcp.Layout(N, I, P), begin, end, src.cuda(), Ps, torch.from_numpy(sbt).cuda(),
                           sbt.shape[1], torch.from_numpy(pos).cuda(), torch.from_numpy(req).cuda(),
                           torch.from_numpy(bt).cuda(), bt.shape[1], arena, pool, status)
    ref = np.zeros(arena.shape, np.uint8)
    for p, b in zip(pos, req):
        o, row = int(olayout.owner(p, N, I)), int(olayout.local_row(p, N, I))
        if begin <= o < end:
            ref[o - begin, bt[b, row // P] * P + row % P] = want[sbt[b, p // Ps] * Ps + p % Ps]
    assert np.array_equal(arena.cpu().numpy(), ref)
    assert int(status.item()) == 0


def test_bad_tokens_are_flagged_and_skipped():
    dcp = _dcp()
    N, P, pool = 2, 8, 3
    lay = dcp.Layout(N, 1, P)
    bt = torch.tensor([[0, 7], [-3, 2]], dtype=torch.int32, device="cuda")
    rows = random_rows(1, 1)
    for p, b, bit in [(-2, 0, 1), (-1, 0, 1), (3, -1, 8), (3, 2, 8), (2 * N * P, 0, 2), (N * P, 0, 4), (0, 1, 4)]:
        arena = torch.zeros(N, pool * P, 416, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (torch.tensor([p], device="cuda"), torch.tensor([b], dtype=torch.int32, device="cuda"), bt, 2)
        dcp.dcp_kv_append_q4(lay, 0, N, rows.cuda(), *args, arena, pool, status)
        assert int(status.item()) == bit, (p, b)
        assert int(arena.count_nonzero()) == 0
        status.zero_()
        kv = torch.full((1, 576), 2.0, dtype=torch.bfloat16, device="cuda")
        dcp.dcp_kv_read_q4(lay, 0, N, arena, pool, *args, kv, status)
        assert int(status.item()) == bit and bool((kv == 2).all())
        # the source side of a relayout: page index past its table, page past its pool
    src = random_rows(16, 2).cuda()
    for sbt, p, bit in [([[0], [0]], 9, 2), ([[2], [0]], 3, 4), ([[-1], [0]], 3, 4)]:
        arena = torch.zeros(N, pool * P, 416, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dcp.dcp_kv_relayout_q4(lay, 0, N, src, 8, torch.tensor(sbt, dtype=torch.int32, device="cuda"), 1,
                               torch.tensor([p], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), bt, 2,
                               arena, pool, status)
        assert int(status.item()) == bit and int(arena.count_nonzero()) == 0


# ---------------------------------------------------------------- partial decode
class Q4State:
    def __init__(self, lens, H, q_len, N, I, P, begin=0, end=None, seed=0, part_dtype=torch.float32, base=0,
                 kv_scale=1.0, max_pages=None, junk=True):
        dcp = _dcp()
        self.lens, self.H, self.q_len, self.N, self.I, self.P, self.base = lens, H, q_len, N, I, P, base
        self.begin, self.end = begin, N if end is None else end
        self.lay = dcp.Layout(N, I, P)
        B, n = len(lens), self.end - self.begin
        self.bt, self.pool = make_tables(lens, N, P, 2, seed + 1, max_pages)
        rows = self.pool * P
        g = torch.Generator().manual_seed(seed + 2)
        kv = (torch.randn(n * rows, 576, generator=g) * kv_scale).to(torch.bfloat16).cuda()
        # rows through the library's own append (checked bit for bit above), one row per position of one request
        one = torch.arange(rows, dtype=torch.int64, device="cuda")
        table = torch.arange(self.pool, dtype=torch.int32, device="cuda")[None]
        self.arena = torch.zeros(n, rows, 416, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for r in range(n):
            dcp.dcp_kv_append_q4(dcp.Layout(1, 1, P), 0, 1, kv[r * rows:(r + 1) * rows], one,
                                 torch.zeros(rows, dtype=torch.int32, device="cuda"), table, self.pool,
                                 self.arena[r:r + 1], self.pool, status)
        assert int(status.item()) == 0
        if junk:
            self.spoil()
        self.values = cache_q4.unpack(self.arena.cpu().numpy())
        self.q = torch.randn(B, q_len, H, 576, generator=g).to(torch.bfloat16)
        self.o = torch.full((n, B, q_len, H, 512), float("nan"), dtype=part_dtype, device="cuda")
        self.lse = torch.full((n, B, q_len, H), float("nan"), device="cuda")
        ws = dcp.dcp_mla_decode_workspace_size_q4(self.lay, self.begin, self.end, B, q_len, H)
        self.ws = torch.empty(ws, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def spoil(self):
        """Every pool row that no request's position uses becomes NaN codes, scales and rope dims."""
        used = np.zeros(tuple(self.arena.shape[:2]), bool)
        for b, S in enumerate(self.lens):
            for r in range(self.begin, self.end):
                rho = np.arange(int(olayout.count(r, S, self.N, self.I)))
                used[r - self.begin, self.bt[b][rho // self.P] * self.P + rho % self.P] = True
        self.arena[torch.from_numpy(~used).cuda()] = 0xFF

    def run(self, stream=None):
        dcp = _dcp()
        dcp.dcp_mla_decode_partial_q4(
            self.lay, self.begin, self.end, self.q.cuda(), self.arena, self.pool, torch.from_numpy(self.bt).cuda(),
            self.bt.shape[1], torch.tensor(self.lens, dtype=torch.int64, device="cuda"), SCALE,
            dcp.DCP_LSE_BASE_2 if self.base else dcp.DCP_LSE_BASE_E, self.o, self.lse, self.ws, self.status, stream)
        torch.cuda.synchronize()

    def check(self, reqs=None, status=0):
        assert int(self.status.item()) == status
        o, lse, q = to_f64(self.o), to_f64(self.lse), to_f64(self.q)
        bf16 = self.o.dtype == torch.bfloat16
        for b in range(len(self.lens)) if reqs is None else reqs:
            S = self.lens[b]
            for r in range(self.begin, self.end):
                n = int(olayout.count(r, S, self.N, self.I))
                rho = np.arange(n)
                K = self.values[r - self.begin, self.bt[b][rho // self.P] * self.P + rho % self.P]
                at = olayout.global_pos(r, rho, self.N, self.I)
                for t in range(self.q_len):
                    seen = K[at <= S - self.q_len + t]
                    ro, rl = attention._softmax_attend(q[b, t], seen, SCALE, 2 if self.base else 0)
                    go, gl = o[r - self.begin, b, t], lse[r - self.begin, b, t]
                    if not len(seen):
                        assert np.all(go == 0) and np.all(np.isneginf(gl))
                        continue
                    x = SCALE * q[b, t] @ seen.T
                    w = np.exp(x - x.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    ds = 576 * 2.0 ** -23 * SCALE * (np.abs(q[b, t]) @ np.abs(seen).T).max(1)
                    tol = (2.0 ** -8 + 2 * ds + 2.0 ** -16)[:, None] * (w @ np.abs(seen[:, :512]))
                    tol = tol + 2.0 ** -110 * np.abs(seen[:, :512]).sum(0)
                    if bf16:
                        tol = tol + 2.0 ** -8 * np.abs(ro)
                    err = np.abs(go - ro)
                    assert np.all(err <= tol), (b, r, t, float((err - tol).max()))
                    assert np.all(np.abs(gl - rl) <= 1.5 * ds + 2.0 ** -20 * np.maximum(1, np.abs(rl))), (b, r, t)


CASES = {
    "tiny": dict(lens=[1024], H=16, q_len=1, N=4, I=1, P=16),
    "one-token": dict(lens=[1], H=1, q_len=1, N=1, I=1, P=8),
    "edges": dict(lens=[1, 2, 3, 4, 5, 63, 64, 65, 127, 128, 129, 511, 513], H=7, q_len=1, N=4, I=1, P=8),
    "h96-base2": dict(lens=[4109, 77, 2000], H=96, q_len=1, N=8, I=1, P=64, base=1),
    "h128": dict(lens=[3000, 1], H=128, q_len=1, N=8, I=1, P=64, part_dtype=torch.bfloat16),
    "verify": dict(lens=[4, 5, 300, 1777], H=128, q_len=4, N=4, I=16, P=64),
    "verify-odd": dict(lens=[3, 1000, 65], H=33, q_len=3, N=3, I=2, P=32, part_dtype=torch.bfloat16),
    "held": dict(lens=[900, 40, 7], H=40, q_len=2, N=6, I=1, P=128, begin=2, end=5),
    "chunk": dict(lens=[700, 64], H=32, q_len=64, N=2, I=1, P=64, base=1),
    "one-shard": dict(lens=[2500, 63], H=64, q_len=1, N=1, I=1, P=256),
    # at most 16 query rows: the other kernel
    "few-verify": dict(lens=[3, 4, 100, 1777], H=5, q_len=3, N=3, I=2, P=32, part_dtype=torch.bfloat16, base=1),
    "few-held": dict(lens=[900, 40, 7], H=8, q_len=2, N=6, I=1, P=128, begin=2, end=5),
    "few-one-shard": dict(lens=[5000, 63], H=16, q_len=1, N=1, I=1, P=256),
    "few-chunk": dict(lens=[700, 64, 65, 16], H=1, q_len=16, N=2, I=1, P=8, base=1),
    "few-long": dict(lens=[40000, 12345], H=15, q_len=1, N=8, I=1, P=64, part_dtype=torch.bfloat16),
    "few-same-request": dict(lens=[9000], H=16, q_len=1, N=16, I=16, P=16),
}


@pytest.mark.parametrize("name", list(CASES))
def test_partial(name):
    st = Q4State(**CASES[name], seed=len(name))
    st.run()
    st.check()
    first = st.o.clone(), st.lse.clone()
    st.run()                                # same bits on a second call
    assert torch.equal(first[0], st.o) and torch.equal(first[1], st.lse)


@pytest.mark.parametrize("H", [24, 6])
@pytest.mark.parametrize("kv_scale", [2.0 ** -6, 8.0])
def test_partial_small_and_large_rows(kv_scale, H):
    """Flat softmax, and one that is almost one key (scores of order 100)."""
    st = Q4State([600, 1300], H, 2, 4, 1, 16, kv_scale=kv_scale, seed=21)
    st.run()
    st.check()


@pytest.mark.parametrize("H", [16, 4])
def test_partial_short_length_and_bad_page(H):
    st = Q4State([50, 2, 400], H, 4, 2, 1, 16, seed=31)
    st.run()                                # request 1 is shorter than q_len: flagged, empty
    assert int(st.status.item()) == 16
    assert bool((st.o[:, 1] == 0).all()) and bool(torch.isneginf(st.lse[:, 1]).all())
    st.check(reqs=[0, 2], status=16)
    st = Q4State([50, 90, 400], 3 * H, 1, 2, 1, 16, seed=32, junk=False)
    st.bt[1, 1] = st.pool
    st.run()
    assert int(st.status.item()) == 4
    st.check(reqs=[0, 2], status=4)
    assert bool(torch.isfinite(st.o).all())


@pytest.mark.parametrize("H", [16, 8])
@pytest.mark.parametrize("length", [2 * 16 * 13 + 1, 2 ** 40, 2 ** 63 - 1])
def test_length_beyond_the_table(length, H):
    """A request that claims more pages than the table has is flagged; the others are right, and it takes no longer."""
    st = Q4State([50, 400, 90], H, 2, 2, 1, 16, seed=33, junk=False)
    assert st.bt.shape[1] == 13
    st.lens = [50, length, 90]
    st.run()
    assert int(st.status.item()) == 4
    st.check(reqs=[0, 2], status=4)


def test_wide_table_and_spare_columns():
    st = Q4State([300, 20], 8, 1, 2, 1, 8, seed=41, max_pages=100)
    st.run()
    st.check()


def test_partial_on_a_side_stream_and_in_a_graph():
    """Captured once, replayed after the queries, the lengths and the cache changed in place."""
    dcp = _dcp()
    st = Q4State([800, 500], 32, 1, 4, 1, 16, seed=51)
    q, bt = st.q.cuda(), torch.from_numpy(st.bt).cuda()
    lens = torch.tensor(st.lens, dtype=torch.int64, device="cuda")

    def call():
        dcp.dcp_mla_decode_partial_q4(st.lay, 0, 4, q, st.arena, st.pool, bt, bt.shape[1], lens, SCALE, 0, st.o,
                                      st.lse, st.ws, st.status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    st.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    st.q = st.q.flip(2).contiguous()
    q.copy_(st.q)
    st.lens = [333, 499]
    lens.copy_(torch.tensor(st.lens))
    st.o.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    st.check()


@pytest.mark.parametrize("H", [16, 8])
def test_two_streams_at_once(H):
    """Two calls in flight on different streams, each with its own workspace and outputs."""
    a = Q4State([3000, 1000], 96, 1, 4, 1, 64, seed=61)
    b = Q4State([2500, 1500, 10], H, 2, 2, 1, 16, seed=62)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    dcp = _dcp()
    held = []
    for st, s in ((a, s1), (b, s2)):
        held.append((st.q.cuda(), torch.from_numpy(st.bt).cuda(),
                     torch.tensor(st.lens, dtype=torch.int64, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, bt, lens), st, s in zip(held, (a, b), (s1, s2)):
            dcp.dcp_mla_decode_partial_q4(st.lay, 0, st.N, q, st.arena, st.pool, bt, bt.shape[1], lens, SCALE, 0,
                                          st.o, st.lse, st.ws, st.status, s)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("H", [16, 24])
def test_rows_past_four_gigabytes(H):
    """Pages at the far end of pools of more than 2^32 bytes in all."""
    dcp = _dcp()
    N, P, pool = 2, 64, 90000                        # 2 x 5.76M rows of 416 bytes: 4.8 GB
    lay = dcp.Layout(N, 1, P)
    arena = torch.zeros(N, pool * P, 416, dtype=torch.uint8, device="cuda")
    S = 300
    bt = torch.tensor([[pool - 1, 5, pool - 2]], dtype=torch.int32, device="cuda")
    rows = random_rows(S, 71)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos, req = torch.arange(S, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_append_q4(lay, 0, N, rows.cuda(), pos, req, bt, 3, arena, pool, status)
    kv = torch.zeros(S, 576, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_read_q4(lay, 0, N, arena, pool, pos, req, bt, 3, kv, status)
    values = cache_q4.unpack(store_rows(rows))
    assert np.array_equal(to_f64(kv), values)
    q = torch.randn(1, 1, H, 576, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    o = torch.empty(N, 1, 1, H, 512, device="cuda")
    lse = torch.empty(N, 1, 1, H, device="cuda")
    ws = torch.empty(dcp.dcp_mla_decode_workspace_size_q4(lay, 0, N, 1, 1, H), dtype=torch.uint8, device="cuda")
    dcp.dcp_mla_decode_partial_q4(lay, 0, N, q.cuda(), arena, pool, bt, 3, torch.tensor([S], device="cuda"), SCALE, 0,
                                  o, lse, ws, status)
    assert int(status.item()) == 0
    for r in range(N):
        K = values[r::N]
        ro, rl = attention._softmax_attend(to_f64(q)[0, 0], K, SCALE, 0)
        ds = 576 * 2.0 ** -23 * SCALE * (np.abs(to_f64(q)[0, 0]) @ np.abs(K).T).max(1)
        x = SCALE * to_f64(q)[0, 0] @ K.T
        w = np.exp(x - rl[:, None])
        assert np.all(np.abs(to_f64(o)[r, 0, 0] - ro) <= (2.0 ** -8 + 2 * ds + 2.0 ** -16)[:, None] * (w @ np.abs(K[:, :512])))
        assert np.all(np.abs(to_f64(lse)[r, 0, 0] - rl) <= ds + 2.0 ** -20 * np.abs(rl))
