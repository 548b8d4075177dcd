"""Padded token lists (pos = req = -1 behind the last token, as dcp_block_tables fills them up) in the calls of the bf16
cache: skipped without a status bit, alone and in a captured serving step; half-padded entries are still flagged."""

import numpy as np
import pytest
import torch

import workloads
from oracle import attention, layout as olayout

from harness import bits, to_f64
from test_gpu_q4 import make_tables

pytestmark = pytest.mark.gpu

SCALE = workloads.SCALE


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def padded_list(lens, seed):
    """Every position of every request, shuffled, with padding among and behind them."""
    pos = np.concatenate([np.arange(n) for n in lens] + [np.full(9, -1)]).astype(np.int64)
    req = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [np.full(9, -1)]).astype(np.int32)
    order = np.random.default_rng(seed).permutation(len(pos))
    return (np.concatenate([pos[order], np.full(21, -1, np.int64)]),
            np.concatenate([req[order], np.full(21, -1, np.int32)]))


@pytest.mark.parametrize("N,I,P,begin,end", [(4, 1, 16, 0, 4), (8, 2, 64, 2, 5), (1, 1, 8, 0, 1)])
def test_slot_map_append_and_relayout(N, I, P, begin, end):
    dcp, lens = _dcp(), [1, 37, 2 * N * P + 5]
    bt, pool = make_tables(lens, N, P, 2, 7)
    sbt, spool = make_tables(lens, 1, 48, 1, 8)
    pos, req = padded_list(lens, 1)
    T, lay, real = len(pos), dcp.Layout(N, I, P), pos >= 0
    d = dict(device="cuda")
    p, r, btd = torch.from_numpy(pos).cuda(), torch.from_numpy(req).cuda(), torch.from_numpy(bt).cuda()
    status = torch.zeros(1, dtype=torch.int32, **d)
    owner, row, slot = (torch.full((T,), 7, dtype=t, **d) for t in (torch.int32, torch.int64, torch.int64))
    dcp.dcp_slot_map(lay, p, r, btd, bt.shape[1], pool, owner, row, slot, status)
    want = olayout.slot_map(pos[real], req[real], bt, N, I, P)
    for got, w in zip((owner, row, slot), (want[0], want[1], want[2])):
        got = got.cpu().numpy()
        assert np.array_equal(got[real], w) and np.all(got[~real] == -1)
    kv = torch.randint(-2 ** 15, 2 ** 15, (T, 576), dtype=torch.int16).view(torch.bfloat16)
    src = torch.randint(-2 ** 15, 2 ** 15, (spool * 48, 576), dtype=torch.int16).view(torch.bfloat16)
    from_src = sbt[req[real], pos[real] // 48] * 48 + pos[real] % 48
    for rows, call in (
            (bits(kv)[real], lambda a: dcp.dcp_kv_append(lay, begin, end, kv.cuda(), p, r, btd, bt.shape[1], a, pool, status)),
            (bits(src)[from_src], lambda a: dcp.dcp_kv_relayout(
                lay, begin, end, src.cuda(), 48, torch.from_numpy(sbt).cuda(), sbt.shape[1], p, r, btd, bt.shape[1], a, pool,
                status))):
        arena = torch.zeros(end - begin, pool * P, 576, dtype=torch.bfloat16, **d)
        call(arena)
        ref = np.zeros(arena.shape, np.uint16)
        mine = (want[0] >= begin) & (want[0] < end)
        ref[want[0][mine] - begin, want[2][mine]] = rows[mine]
        assert np.array_equal(bits(arena), ref)
    assert int(status.item()) == 0


@pytest.mark.parametrize("p,b,bit", [(-1, 0, 1), (-2, -1, 1), (0, -1, 8)])
def test_half_padded_entries_are_flagged(p, b, bit):
    dcp, d = _dcp(), dict(device="cuda")
    lay, bt = dcp.Layout(2, 1, 8), torch.zeros(1, 1, dtype=torch.int32, **d)
    pos, req = torch.tensor([p], **d), torch.tensor([b], dtype=torch.int32, **d)
    rows = torch.ones(8, 576, dtype=torch.bfloat16, **d)
    out = [torch.zeros(1, dtype=t, **d) for t in (torch.int32, torch.int64, torch.int64)]
    for call in (lambda st, ar: dcp.dcp_slot_map(lay, pos, req, bt, 1, 1, *out, st),
                 lambda st, ar: dcp.dcp_kv_append(lay, 0, 2, rows[:1], pos, req, bt, 1, ar, 1, st),
                 lambda st, ar: dcp.dcp_kv_relayout(lay, 0, 2, rows, 8, bt, 1, pos, req, bt, 1, ar, 1, st)):
        st, ar = torch.zeros(1, dtype=torch.int32, **d), torch.zeros(2, 8, 576, dtype=torch.bfloat16, **d)
        call(st, ar)
        assert int(st.item()) == bit and int(ar.count_nonzero()) == 0


def test_a_bf16_serving_step_in_one_graph():
    """Tables, append of the padded lists, partials and merge captured once; replayed with other lengths and rows."""
    from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
    dcp = _dcp()
    B, H, N, I, P, T = 4, 16, 2, 1, 16, 96
    lay = dcp.Layout(N, I, P)
    tab = BlockTables(lay, B, pool_pages=24, max_pages=8, max_tokens=T)
    dec = ShardedMlaDecoder(lay, B, 1, H, 24, 8, SCALE, 0, torch.float32)
    new = torch.zeros(B, dtype=torch.int64, device="cuda")
    rows = torch.zeros(T, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, 1, H, 576, dtype=torch.bfloat16, device="cuda")

    def step():
        pos, req = tab.update(new)
        dec.append(rows, pos, req, tab.block_table)
        return dec.decode(q, tab.block_table, tab.seq_lens)

    step()                                          # nothing yet: padding only, requests of length 0 (flagged)
    assert dec.status_bits() == 16
    dec.status.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    g = torch.Generator().manual_seed(111)
    held = [np.zeros((0, 576)) for _ in range(B)]
    for lens in ([20, 1, 33, 40], [21, 2, 34, 41], [21, 60, 1, 42], [90, 61, 2, 43]):
        r, qs = (torch.randn(*x, generator=g).to(torch.bfloat16) for x in ((T, 576), (B, 1, H, 576)))
        rows.copy_(r)
        q.copy_(qs)
        new.copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        n = 0
        for b, S in enumerate(lens):
            k = max(0, S - len(held[b]))
            held[b] = np.concatenate([held[b][:S], to_f64(r)[n:n + k]])
            n += k
            K, x = held[b], SCALE * to_f64(qs)[b, 0] @ held[b].T
            ro, rl = attention._softmax_attend(to_f64(qs)[b, 0], K, SCALE, 0)
            # the partial's bounds (test_gpu_q4.py; the products are the same), and the merge's two fp32 roundings a shard
            ds = 576 * 2.0 ** -23 * SCALE * (np.abs(to_f64(qs)[b, 0]) @ np.abs(K).T).max(1)
            tol = (2.0 ** -8 + 4 * ds + 2.0 ** -15)[:, None] * (np.exp(x - rl[:, None]) @ np.abs(K[:, :512]))
            assert np.all(np.abs(to_f64(o)[b, 0] - ro) <= tol)
            assert np.all(np.abs(to_f64(lse)[b, 0] - rl) <= 2 * ds + 2.0 ** -19 * np.maximum(1, np.abs(rl)))
    assert tab.status_bits() == 0 and dec.status_bits() == 0
