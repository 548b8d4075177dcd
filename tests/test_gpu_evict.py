"""Eviction on the GPU: the rows that stay (exact), their move in place (bit for bit), and a serving run on both caches."""

import numpy as np
import pytest
import torch

from oracle import evict, layout as olayout

from test_gpu_q4 import make_tables

pytestmark = pytest.mark.gpu


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def make_weights(n, B, W, seed, plain=False):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal((n, B, W))).astype(np.float32)
    if plain:
        return w
    w[w < 0.3] = 0.0
    w[rng.random(w.shape) < 0.05] = -0.0
    some = rng.random(w.shape) < 0.3
    w[some] = np.round(w[some])
    w[rng.random(w.shape) < 0.02] = np.nan
    w[rng.random(w.shape) < 0.02] = np.inf
    w[rng.random(w.shape) < 0.02] = -np.inf
    w[rng.random(w.shape) < 0.03] *= -1
    w[rng.random(w.shape) < 0.01] = np.float32(1e-42)          # below the normal range
    return w


def run_select(w, lens, new, N, I, P, begin, end, sinks, recent, room=None):
    dcp = _dcp()
    n, B = end - begin, len(lens)
    room = room or max(1, max(int(olayout.count(0, x, N, I)) for x in new)) + 3
    kept = torch.full((n, B, room), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_evict_select(dcp.Layout(N, I, P), begin, end, torch.tensor(lens, dtype=torch.int64, device="cuda"),
                         torch.tensor(new, dtype=torch.int64, device="cuda"), sinks, recent, torch.from_numpy(w).cuda(), kept, status)
    return kept.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("lens,new,N,I,P,begin,end", [
    ([1], [1], 1, 1, 8, 0, 1), ([1], [0], 1, 1, 8, 0, 1), ([100, 3, 0, 777], [50, 1, 0, 776], 4, 1, 16, 0, 4),
    ([1000, 999], [333, 998], 3, 8, 8, 1, 3), ([5000], [4000], 1, 1, 64, 0, 1), ([20000, 31], [123, 31], 2, 2, 16, 0, 2),
    ([33] * 90, [32] * 90, 8, 1, 8, 0, 8)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 16), (1000, 0), (0, 100000), (3, 60)])
def test_select(lens, new, N, I, P, begin, end, sinks, recent):
    W = max(1, int(olayout.count(0, max(lens), N, I))) + 5
    w = make_weights(end - begin, len(lens), W, 3)
    kept, status = run_select(w, lens, new, N, I, P, begin, end, sinks, recent)
    assert status == 0
    for r in range(begin, end):
        for b, S in enumerate(lens):
            want = evict.select(w[r - begin, b], r, S, new[b], N, I, sinks, recent)
            got = kept[r - begin, b]
            assert got[:len(want)].tolist() == want, (r, b)
            assert np.all(got[len(want):] == -7)


@pytest.mark.parametrize("n,m", [(200001, 100000), (200001, 200000), (131072, 1), (65536, 65535)])
@pytest.mark.parametrize("alike", [False, True])
def test_select_of_a_long_unit(n, m, alike):
    """One shard of many rows, against a stable sort; with weights that are nearly all alike."""
    rng = np.random.default_rng(5)
    w = (rng.integers(0, 3, n) if alike else rng.random(n)).astype(np.float32)[None, None]
    kept, status = run_select(w, [n], [m], 1, 1, 16, 0, 1, 10, 500)
    assert status == 0
    nr = min(500, m - min(10, m))
    mid = np.argsort(-w[0, 0, 10:n - 500], kind="stable")[:max(0, m - 10 - nr)] + 10
    want = np.sort(np.concatenate([np.arange(min(10, m)), mid, np.arange(n - nr, n)]))
    assert np.array_equal(kept[0, 0, :m], want)


def test_select_refusals_on_the_device():
    w = make_weights(2, 5, 50, 1, plain=True)
    lens, new = [90, 40, 101, 80, 60], [91, -1, 10, 80, 59]
    kept, status = run_select(w, lens, new, 2, 1, 8, 0, 2, 0, 0, room=35)
    assert status == 16
    assert np.all(kept[:, 0] == -1) and np.all(kept[:, 1] == -7)             # longer than it is: 46 rows; none
    assert np.all(kept[0, 2, :5] == -1) and np.all(kept[0, 2, 5:] == -7)     # shard 0 has 51 rows of 101, more than 50
    assert kept[1, 2, :5].tolist() == evict.select(w[1, 2], 1, 101, 10, 2, 1, 0, 0)
    assert np.all(kept[:, 3] == -1)                                          # 40 rows do not fit 35 entries
    for r in range(2):
        want = evict.select(w[r, 4], r, 60, 59, 2, 1, 0, 0)
        assert kept[r, 4, :len(want)].tolist() == want


# ---------------------------------------------------------------- compact
def run_compact(q4, arena, kept, new, bt, pool, N, I, P, begin, end, weights=None, stream=None):
    dcp = _dcp()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = dcp.dcp_kv_compact_q4 if q4 else dcp.dcp_kv_compact
    fn(dcp.Layout(N, I, P), begin, end, torch.from_numpy(kept).cuda(), torch.tensor(new, dtype=torch.int64, device="cuda"),
       torch.from_numpy(bt).cuda(), bt.shape[1], arena, pool, status, weights=weights, stream=stream)
    return int(status.item())


def random_arena(q4, n, rows, seed):
    g = torch.Generator().manual_seed(seed)
    if q4:
        return torch.randint(0, 256, (n, rows, 416), dtype=torch.uint8, generator=g)
    return torch.randint(-32768, 32768, (n, rows, 576), dtype=torch.int16, generator=g)   # NaN patterns too


def moved(arena, weights, kept, new, bt, N, I, P, begin, end):
    """The oracle's move: every row from before the call."""
    a, w = arena.copy(), None if weights is None else weights.copy()
    for r in range(begin, end):
        for b in range(len(new)):
            for i in range(int(olayout.count(r, new[b], N, I))):
                k = int(kept[r - begin, b, i])
                if k < i:
                    continue
                a[r - begin, bt[b, i // P] * P + i % P] = arena[r - begin, bt[b, k // P] * P + k % P]
                if w is not None:
                    w[r - begin, b, i] = weights[r - begin, b, k]
    return a, w


def random_kept(lens, new, N, I, begin, end, seed, how):
    rng = np.random.default_rng(seed)
    room = max(1, max(int(olayout.count(0, x, N, I)) for x in new)) + 2
    kept = np.full((end - begin, len(lens), room), -1, np.int32)
    for r in range(begin, end):
        for b, S in enumerate(lens):
            n, m = int(olayout.count(r, S, N, I)), int(olayout.count(r, new[b], N, I))
            if how == "ascending":
                k = np.sort(rng.permutation(n)[:m])
            elif how == "identity":
                k = np.arange(m)
            elif how == "shifted":                             # every row one on: a chain through the whole unit
                k = np.minimum(np.arange(m) + 1, n - 1)
            else:                                              # any row not before its place, repeats and skips among them
                k = rng.integers(np.arange(m), n) if m else np.zeros(0, int)
                k[rng.random(m) < 0.1] = -1
            kept[r - begin, b, :m] = k
    return kept


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("how", ["ascending", "identity", "shifted", "any"])
@pytest.mark.parametrize("lens,new,N,I,P,begin,end", [
    ([1], [1], 1, 1, 8, 0, 1), ([700, 1, 0, 64], [699, 1, 0, 10], 4, 1, 16, 0, 4), ([400, 333], [100, 332], 3, 6, 6, 1, 3),
    ([3000], [1500], 1, 1, 3, 0, 1), ([9000, 50], [7000, 49], 2, 1, 64, 0, 2), ([100] * 80, [60] * 80, 8, 1, 8, 0, 8)])
def test_compact(q4, how, lens, new, N, I, P, begin, end):
    bt, pool = make_tables(lens, N, P, 3, 4)
    arena = random_arena(q4, end - begin, pool * P, 2)
    kept = random_kept(lens, new, N, I, begin, end, 6, how)
    W = bt.shape[1] * P
    weights = np.random.default_rng(1).random((end - begin, len(lens), W)).astype(np.float32)
    want, want_w = moved(arena.numpy(), weights, kept, new, bt, N, I, P, begin, end)
    dev, dw = arena.cuda(), torch.from_numpy(weights).cuda()
    view = dev if q4 else dev.view(torch.bfloat16)
    assert run_compact(q4, view, kept, new, bt, pool, N, I, P, begin, end, dw) == 0
    assert np.array_equal(dev.cpu().numpy(), want) and np.array_equal(dw.cpu().numpy(), want_w)
    dev = arena.cuda()
    assert run_compact(q4, dev if q4 else dev.view(torch.bfloat16), kept, new, bt, pool, N, I, P, begin, end) == 0
    assert np.array_equal(dev.cpu().numpy(), want)


@pytest.mark.parametrize("q4", [False, True])
def test_compact_of_bad_entries(q4):
    N, I, P = 1, 1, 4
    bt = np.array([[2, 0, 9, 3], [1, 4, 5, -1]], np.int32)     # request 0's third page lies outside the pool
    arena = random_arena(q4, 1, 6 * P, 8)
    kept = np.array([[[3, 5, 1, 8, 4, 12, 16, 15], [-1, 2, -2, 3, 100, 5, 6, 7]]], np.int32)
    weights = np.arange(2 * 15, dtype=np.float32).reshape(1, 2, 15)
    dev, dw = arena.cuda(), torch.from_numpy(weights).cuda()
    status = run_compact(q4, dev if q4 else dev.view(torch.bfloat16), kept, [8, 5], bt, 6, N, I, P, 0, 1, dw)
    assert status == 1 | 2 | 4                                  # below their place; past the table or the weights; bad page
    want, w = arena.numpy().copy(), weights.copy()
    at = lambda b, i: bt[b, i // P] * P + i % P                 # noqa: E731
    for b, i, k in ((0, 0, 3), (0, 1, 5), (0, 5, 12), (1, 1, 2)):
        want[0, at(b, i)] = arena.numpy()[0, at(b, k)]
        w[0, b, i] = weights[0, b, k]
    assert np.array_equal(dev.cpu().numpy(), want) and np.array_equal(dw.cpu().numpy(), w)
    dev = arena.cuda()
    status = run_compact(q4, dev if q4 else dev.view(torch.bfloat16), kept, [9, -1], bt, 6, N, I, P, 0, 1)
    assert status == 16 and np.array_equal(dev.cpu().numpy(), arena.numpy())   # more rows than entries; a negative length


def test_compact_beyond_four_gigabytes_on_another_stream():
    P, pages = 64, 60000
    bt = np.array([[59999, 1, 59990, 58300]], np.int32)
    arena = torch.zeros(1, pages * P, 576, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(256, 576, device="cuda").to(torch.bfloat16)
    at = torch.from_numpy(bt[0, np.arange(256) // P].astype(np.int64) * P + np.arange(256) % P).cuda()
    arena[0, at] = rows
    kept = np.sort(np.random.default_rng(3).permutation(256)[:200]).astype(np.int32)[None, None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    dcp = _dcp()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, new, table = torch.from_numpy(kept).cuda(), torch.tensor([200], device="cuda"), torch.from_numpy(bt).cuda()
    torch.cuda.synchronize()
    dcp.dcp_kv_compact(dcp.Layout(1, 1, P), 0, 1, k, new, table, 4, arena, pages, status, stream=side)
    side.synchronize()
    want = rows.clone()
    want[:200] = rows[k[0, 0].long()]
    assert int(status.item()) == 0 and torch.equal(arena[0, at], want)


@pytest.mark.parametrize("value", [float("-inf"), -3e38, float("nan"), 0.0])
@pytest.mark.parametrize("keep", [1, 700, 999, 1000])
def test_select_of_equal_weights(value, keep):
    w = np.full((1, 1, 1000), value, np.float32)
    kept, status = run_select(w, [1000], [keep], 1, 1, 8, 0, 1, 0, 0)
    assert status == 0 and kept[0, 0, :keep].tolist() == list(range(keep))
