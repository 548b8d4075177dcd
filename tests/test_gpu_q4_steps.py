"""The 4-bit cache where its softmax, its work split and its callers can go wrong: jumping maxima, many short
requests, the row limit, several ranks, several threads, one graph for a whole serving step.

Bounds are those of the partial decode's tests; a merge adds two fp32 roundings a shard (below 2^-16 of
sum_p w_p |v_p|), and a bf16 exchange rounds each shard's partial once more (2^-8 of it)."""

import threading

import numpy as np
import pytest
import torch

import workloads
from oracle import attention, cache_q4

from harness import to_f64
from test_gpu_q4 import Q4State, SCALE, make_tables, random_rows, store_rows

pytestmark = pytest.mark.gpu


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def plant(st, b, at, rows):
    """Rows of request b at positions `at` (one held shard of one) into the arena and the oracle's copy."""
    packed = store_rows(rows)
    slot = st.bt[b][np.asarray(at) // st.P] * st.P + np.asarray(at) % st.P
    st.arena[0, torch.from_numpy(slot.astype(np.int64)).cuda()] = torch.from_numpy(packed).cuda()
    st.values[0, slot] = cache_q4.unpack(packed)


# (position, factor): scores of about 40 |factor| e-units in tiles of 64 keys, whose halves of 32 belong to the two
# CTAs of a pair: the maximum is raised by one half, then by the other, in the same tile and in the next, and falls
JUMPS = {
    "up": [(5, 0.5), (40, 1.0), (64, 1.5), (100, 2.0), (3000, 4.0), (3040, 6.0), (9001, 8.0)],
    "up-other-half": [(40, 0.5), (5 + 64, 1.0), (96 + 64, 1.5), (64 + 64, 2.0), (3040, 4.0), (3064, 6.0), (9050, 8.0)],
    "down": [(0, 8.0), (32, 7.0), (64, 6.0), (130, 4.0), (5000, 2.0)],
    "from-below": [(i, -8.0) for i in range(128)] + [(i, -4.0) for i in range(128, 192)] + [(4000, 1.0)],
    "ends-with-it": [(10299, 6.0)],
}


@pytest.mark.parametrize("H,q_len", [(96, 1), (16, 1), (40, 3)])
@pytest.mark.parametrize("name", list(JUMPS))
def test_running_max_jumps(name, H, q_len):
    lens = [10300, 3041, 129]                       # cut behind different jumps
    st = Q4State(lens, H, q_len, 1, 1, 64, seed=81, kv_scale=0.5, base=1)
    g = torch.Generator().manual_seed(82)
    base = torch.randn(len(lens), 1, 1, 576, generator=g)
    st.q = (base + torch.randn(len(lens), q_len, H, 576, generator=g) / 8).to(torch.bfloat16)
    for b, S in enumerate(lens):
        at = [(p, f) for p, f in JUMPS[name] if p < S]
        if at:
            plant(st, b, [p for p, _ in at], torch.cat([base[b, 0] * f for _, f in at]).to(torch.bfloat16))
    st.run()
    st.check()


@pytest.mark.parametrize("H", [16, 17])
def test_many_short_requests(H):
    """More units of work than pairs of CTAs, most of one tile or of none."""
    lens = [int(x) for x in np.random.default_rng(91).integers(1, 140, size=700)]
    st = Q4State(lens, H, 1, 4, 1, 8, seed=92)
    st.run()
    st.check()


def test_row_limit():
    """512 x 128 query rows, the most a call takes, causal over 700 positions."""
    st = Q4State([700], 128, 512, 4, 1, 16, seed=93)
    st.run()
    st.check()


def reference(q, seen, base=0):
    """fp64 attention of q [H, 576] over rows [n, 576], the bounds of its partial's o and lse, and sum_p w_p |v_p|."""
    ro, rl = attention._softmax_attend(q, seen, SCALE, base)
    x = SCALE * q @ seen.T
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    ds = 576 * 2.0 ** -23 * SCALE * (np.abs(q) @ np.abs(seen).T).max(1)
    wv = w @ np.abs(seen[:, :512])
    return ro, rl, (2.0 ** -8 + 4 * ds + 2.0 ** -15)[:, None] * wv, 2 * ds + 2.0 ** -19 * np.maximum(1, np.abs(rl)), wv


@pytest.mark.parametrize("world,strategy,wire", [(4, "a2a", torch.bfloat16), (2, "a2a", torch.float32),
                                                 (4, "ag_rs", torch.float32)])
def test_ranks_with_4_bit_pools(world, strategy, wire):
    """Each rank appends what it owns and runs its shards' partials; the exchange as device copies."""
    from context_sharded_mla_gb300.group import DcpGroupDecoder
    dcp = _dcp()
    N, I, P, H, B = 4, 1, 16, 32, 3
    lens = [500, 3, 777]
    bt, pool = make_tables(lens, N, P, 1, 95)
    btd, seq = torch.from_numpy(bt).cuda(), torch.tensor(lens, device="cuda")
    rows = [random_rows(n, 96 + b) for b, n in enumerate(lens)]
    kv = torch.cat(rows).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    req = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(lens)]).cuda()
    q = torch.randn(B, 1, H, 576, generator=torch.Generator().manual_seed(97)).to(torch.bfloat16)
    ranks = [DcpGroupDecoder(dcp.Layout(N, I, P), B, 1, H, pool, bt.shape[1], SCALE, w, world, 0, strategy, wire,
                             torch.float32, cache="q4") for w in range(world)]
    for r in ranks:
        r.append(kv, pos, req, btd)
        r.local.partial(q.cuda(), btd, seq)
        if strategy == "a2a":
            dcp.dcp_pack_partials(r.local.o_part, r.local.lse_part, world, r.xchg.send, wire)
    if strategy == "a2a":
        for d, rd in enumerate(ranks):
            for w, rw in enumerate(ranks):
                rd.xchg.recv[w].copy_(rw.xchg.send[d])
        for r in ranks:
            x = r.xchg
            dcp.dcp_lse_merge_packed(x.recv, world, x.n_held, x.lse_base, x.o.view(-1, 512), x.lse.view(-1), wire)
    else:
        lse_all = torch.cat([r.local.lse_part for r in ranks]).view(N, -1, H)
        for r in ranks:
            x = r.xchg
            dcp.dcp_lse_rescale(lse_all, r.local.o_part, x.shard_begin, world, x.lse_base, x.o_sum, x.lse_blocks)
        for d, rd in enumerate(ranks):
            rd.xchg.o.copy_(torch.stack([rw.xchg.o_sum[d] for rw in ranks]).sum(0))
    torch.cuda.synchronize()
    for r in ranks:
        assert r.status_bits() == 0
        h0, h1 = r.head_begin, r.head_end
        o, lse = to_f64(r.xchg.o).reshape(B, h1 - h0, 512), to_f64(r.xchg.lse).reshape(B, h1 - h0)
        for b in range(B):
            ro, rl, tol, tol_lse, wv = reference(to_f64(q[b, 0, h0:h1]), cache_q4.unpack(store_rows(rows[b])))
            if wire == torch.bfloat16:
                tol = tol + 2.0 ** -8 * wv
            assert np.all(np.abs(o[b] - ro) <= tol)
            assert np.all(np.abs(lse[b] - rl) <= tol_lse)


def test_two_threads():
    """Two host threads, each with its own stream, cache and workspace."""
    states = [Q4State([2000, 31], 48, 1, 2, 1, 64, seed=101), Q4State([900, 1500, 4], 16, 4, 4, 1, 16, seed=102)]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def work(st):
        try:
            stream = torch.cuda.Stream()
            start.wait(timeout=60)
            with torch.cuda.stream(stream):
                for _ in range(4):
                    st.run(stream)
        except Exception as e:   # reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(st,)) for st in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    for st in states:
        st.check()


def test_a_serving_step_in_one_graph():
    """Tables, append, read back, partials and merge captured once; replayed with other lengths, rows and queries."""
    from context_sharded_mla_gb300.step import BlockTables, ShardedMlaDecoder
    dcp = _dcp()
    B, H, N, I, P, T = 4, 16, 2, 1, 16, 96
    lay = dcp.Layout(N, I, P)
    tab = BlockTables(lay, B, pool_pages=24, max_pages=8, max_tokens=T)
    dec = ShardedMlaDecoder(lay, B, 1, H, 24, 8, SCALE, 0, torch.float32, cache="q4")
    new = torch.zeros(B, dtype=torch.int64, device="cuda")
    rows = torch.zeros(T, 576, dtype=torch.bfloat16, device="cuda")
    back = torch.zeros(T, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, 1, H, 576, dtype=torch.bfloat16, device="cuda")

    def step():
        pos, req = tab.update(new)
        dec.append(rows, pos, req, tab.block_table)
        dcp.dcp_kv_read_q4(lay, 0, N, dec.arena, 24, pos, req, tab.block_table, 8, back, dec.status)
        return dec.decode(q, tab.block_table, tab.seq_lens)

    step()                                          # nothing yet: no token, requests of length 0 (flagged)
    assert dec.status_bits() == 16
    dec.status.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    g = torch.Generator().manual_seed(111)
    held = [np.zeros((0, 576)) for _ in range(B)]
    for lens in ([20, 1, 33, 40], [21, 2, 34, 41], [21, 60, 1, 42], [90, 61, 2, 43]):
        r = torch.randn(T, 576, generator=g).to(torch.bfloat16)
        qs = torch.randn(B, 1, H, 576, generator=g).to(torch.bfloat16)
        rows.copy_(r)
        q.copy_(qs)
        new.copy_(torch.tensor(lens))
        back.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        values = cache_q4.unpack(store_rows(r))
        n = 0
        for b, S in enumerate(lens):
            k = max(0, S - len(held[b]))
            held[b] = np.concatenate([held[b][:S], values[n:n + k]])
            n += k
        assert np.array_equal(to_f64(back)[:n], values[:n]) and bool((back[n:] == 5.0).all())
        for b in range(B):
            ro, rl, tol, tol_lse, _ = reference(to_f64(qs)[b, 0], held[b])
            assert np.all(np.abs(to_f64(o)[b, 0] - ro) <= tol)
            assert np.all(np.abs(to_f64(lse)[b, 0] - rl) <= tol_lse)
    assert tab.status_bits() == 0 and dec.status_bits() == 0


def test_read_of_repeated_and_foreign_tokens():
    """The same token many times, another shard's, padding: rows that are not held stay as they were."""
    dcp = _dcp()
    N, P, S = 3, 8, 50
    lay = dcp.Layout(N, 1, P)
    bt, pool = make_tables([S], N, P, 1, 121)
    rows = random_rows(S, 122)
    arena = torch.zeros(2, pool * P, 416, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    btd = torch.from_numpy(bt).cuda()
    dcp.dcp_kv_append_q4(lay, 1, 3, rows.cuda(), torch.arange(S, device="cuda"),
                         torch.zeros(S, dtype=torch.int32, device="cuda"), btd, bt.shape[1], arena, pool, status)
    pos = torch.from_numpy(np.random.default_rng(123).integers(0, S, size=5001))
    pos[::7] = -1
    req = torch.where(pos < 0, -1, 0).to(torch.int32)
    kv = torch.full((5001, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_read_q4(lay, 1, 3, arena, pool, pos.cuda(), req.cuda(), btd, bt.shape[1], kv, status)
    want = np.full((5001, 576), 3.0)
    mine = ((pos >= 0) & (pos % N != 0)).numpy()
    want[mine] = cache_q4.unpack(store_rows(rows))[pos.numpy()[mine]]
    assert int(status.item()) == 0 and np.array_equal(to_f64(kv), want)


def test_tensors_that_do_not_fit():
    """Types, shapes, strides and places are named before anything is launched."""
    dcp = _dcp()
    lay = dcp.Layout(2, 1, 16)
    d = dict(device="cuda")
    arena = torch.zeros(2, 32, 416, dtype=torch.uint8, **d)
    kv, pos = torch.zeros(3, 576, dtype=torch.bfloat16, **d), torch.zeros(3, dtype=torch.int64, **d)
    req, bt, st = torch.zeros(3, dtype=torch.int32, **d), torch.zeros(1, 2, dtype=torch.int32, **d), torch.zeros(
        1, dtype=torch.int32, **d)
    ok = dict(kv=kv, pos=pos, req=req, bt=bt, arena=arena, status=st)

    def refused(match, **kw):
        a = dict(ok, **kw)
        with pytest.raises(ValueError, match=match):
            dcp.dcp_kv_append_q4(lay, 0, 2, a["kv"], a["pos"], a["req"], a["bt"], 2, a["arena"], 2, a["status"])

    refused("kv_new must be torch.bfloat16", kv=kv.float())
    refused("kv_new must have shape", kv=kv[:2].contiguous())
    refused("pos must be torch.int64", pos=pos.int())
    refused("req must have shape", req=req[:2])
    refused("block_table must be contiguous", bt=torch.zeros(1, 4, dtype=torch.int32, **d)[:, ::2])
    refused("arena must have shape", arena=arena[:1])
    refused("arena must be torch.uint8", arena=torch.zeros(2, 32, 576, dtype=torch.bfloat16, **d))
    refused("status must be a CUDA tensor", status=st.cpu())
    with pytest.raises(dcp.DcpError):
        dcp.dcp_kv_append_q4(lay, 0, 2, kv, pos, req, bt, 3, arena, 2, st)      # more pages than the table has columns
    q = torch.zeros(1, 1, 4, 576, dtype=torch.bfloat16, **d)
    o, lse, S = torch.zeros(2, 1, 1, 4, 512, **d), torch.zeros(2, 1, 1, 4, **d), torch.zeros(1, dtype=torch.int64, **d)
    with pytest.raises(dcp.DcpError):                                            # no workspace
        dcp.dcp_mla_decode_partial_q4(lay, 0, 2, q, arena, 2, bt, 2, S, SCALE, 0, o, lse, None, st)
    with pytest.raises(ValueError):
        dcp.dcp_mla_decode_partial_q4(lay, 0, 2, q, arena, 2, bt, 2, S, SCALE, 0, o.half(), lse, None, st)
    with pytest.raises(dcp.DcpError):                                            # seq_lens is new_lens
        dcp.dcp_block_tables(lay, S, S, bt, 2, req, torch.tensor([0, 3], **d), torch.zeros(2, dtype=torch.int64, **d), st)
    assert int(st.item()) == 0
