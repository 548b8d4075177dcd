"""NaN in the partials and in visible cached rows: it reaches the output of the rows that see it, in o and lse, and
leaves every other row's bits as they are without it.  (A part whose lse is NaN is not an empty part.)"""

import pytest
import torch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


# ---------------------------------------------------------------- merges
def parts(n, T, H, dtype, seed):
    """Partials of n shards, with empty parts, and copies with NaN at the rows returned as a mask [T, H]."""
    g = torch.Generator().manual_seed(seed)
    o = torch.randn(n, T, H, 512, generator=g).to(dtype)
    lse = torch.randn(n, T, H, generator=g) * 3
    if n > 1:
        empty = torch.rand(n, T, H, generator=g) < 0.2
        o[empty], lse[empty] = 0, -INF
    lse[:, 3, 1], o[:, 3, 1] = -INF, 0              # a row without a key
    o2, lse2 = o.clone(), lse.clone()
    bad = torch.zeros(T, H, dtype=torch.bool)
    for t, h, r in [(0, 0, 0), (1, H - 1, n - 1), (T - 1, 0, n // 2)]:
        lse2[r, t, h], o2[r, t, h] = NAN, NAN
        bad[t, h] = True
    lse2[:, 2, 0], o2[:, 2, 0] = -INF, 0            # the other parts empty
    lse2[n - 1, 2, 0], o2[n - 1, 2, 0] = NAN, NAN
    bad[2, 0] = True
    lse2[:, T - 1, H - 1], o2[:, T - 1, H - 1] = NAN, NAN   # all of them NaN
    bad[T - 1, H - 1] = True
    return o, lse, o2, lse2, bad


def compare(clean, got, bad):
    """Outputs [T, H, ...]: NaN where bad, the clean run's bits elsewhere."""
    bad = bad.to(got.device)
    assert bool(torch.isnan(got[bad]).all())
    assert torch.equal(clean[~bad], got[~bad])


@pytest.mark.parametrize("base", [0, 1])
@pytest.mark.parametrize("n", [1, 2, 5, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_merge(n, dtype, base):
    dcp, (T, H) = _dcp(), (9, 4)
    o, lse, o2, lse2, bad = parts(n, T, H, dtype, 10 * n + base)
    outs = []
    for a, b in ((o, lse), (o2, lse2)):
        m, l = torch.zeros(T * H, 512, device="cuda"), torch.zeros(T * H, device="cuda")
        dcp.dcp_lse_merge(a.view(n, -1, 512).cuda(), b.view(n, -1).cuda(), base, m, l)
        outs.append((m.view(T, H, 512), l.view(T, H)))
    for clean, got in zip(*outs):
        compare(clean, got, bad)


@pytest.mark.parametrize("base", [0, 1])
@pytest.mark.parametrize("wire", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("world,held", [(1, 3), (2, 1), (4, 2)])
def test_merge_packed(world, held, wire, base):
    dcp, (T, H) = _dcp(), (6, 8)
    n, Hd = world * held, 8 // world
    outs = []
    o, lse, o2, lse2, bad = parts(n, T, H, torch.float32, n)
    for a, b in ((o, lse), (o2, lse2)):
        chunk = dcp.dcp_a2a_chunk_bytes(held, T, H, world, wire)
        sends = []
        for w in range(world):
            send = torch.zeros(world, chunk, dtype=torch.uint8, device="cuda")
            dcp.dcp_pack_partials(a[w * held:(w + 1) * held].contiguous().cuda(),
                                  b[w * held:(w + 1) * held].contiguous().cuda(), world, send, wire)
            sends.append(send)
        ms, ls = [], []
        for d in range(world):
            recv = torch.stack([s[d] for s in sends]).contiguous()
            m, l = torch.zeros(T * Hd, 512, device="cuda"), torch.zeros(T * Hd, device="cuda")
            dcp.dcp_lse_merge_packed(recv, world, held, base, m, l, wire)
            ms.append(m.view(T, Hd, 512))
            ls.append(l.view(T, Hd))
        outs.append((torch.cat(ms, 1), torch.cat(ls, 1)))
    for clean, got in zip(*outs):
        compare(clean, got, bad)


@pytest.mark.parametrize("base", [0, 1])
@pytest.mark.parametrize("world,held", [(1, 3), (2, 1), (4, 2)])
def test_rescale(world, held, base):
    """The ranks' blocks added up, as the reduce-scatter does."""
    dcp, (T, H) = _dcp(), (6, 8)
    n, Hd = world * held, 8 // world
    outs = []
    o, lse, o2, lse2, bad = parts(n, T, H, torch.float32, n)
    for a, b in ((o, lse), (o2, lse2)):
        total, ls = torch.zeros(world, T, Hd, 512, device="cuda"), []
        for w in range(world):
            o_sum, l = torch.zeros(world, T, Hd, 512, device="cuda"), torch.zeros(world, T, Hd, device="cuda")
            dcp.dcp_lse_rescale(b.cuda(), a[w * held:(w + 1) * held].contiguous().cuda(), w * held, world, base, o_sum, l)
            total += o_sum
            ls.append(l)
        assert all(torch.equal(ls[0].nan_to_num(7.0), x.nan_to_num(7.0)) for x in ls)
        outs.append((total.permute(1, 0, 2, 3).reshape(T, H, 512), ls[0].permute(1, 0, 2).reshape(T, H)))
    for clean, got in zip(*outs):
        compare(clean, got, bad)


@pytest.mark.parametrize("base", [0, 1])
@pytest.mark.parametrize("n,T,H", [(1, 9, 3), (8, 40, 4), (64, 20, 2)])
def test_merge_absorb(n, T, H, base):
    dcp = _dcp()
    w_vc = torch.randn(H, 512, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    o, lse, o2, lse2, bad = parts(n, T, H, torch.float32, n + T)
    outs = []
    for a, b in ((o, lse), (o2, lse2)):
        v, l = torch.zeros(T, H, 128, device="cuda"), torch.zeros(T, H, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dcp.dcp_lse_merge_absorb_o(a.cuda(), b.cuda(), base, w_vc, v, l, status)
        assert int(status.item()) == 0
        outs.append((v, l))
    for clean, got in zip(*outs):
        compare(clean, got, bad)


# ---------------------------------------------------------------- partial decodes
def runs(st, spoil):
    """(o, lse) of a Q4State without and with what `spoil` writes into its arena or query."""
    out = []
    for bad in (False, True):
        if bad:
            spoil(st)
        st.o.fill_(5.0)
        st.lse.fill_(5.0)
        st.run()
        assert int(st.status.item()) == 0
        out.append((st.o.clone(), st.lse.clone()))
    return out


def slot_of(st, b, p):
    """(held shard, pool row) of position p of request b."""
    from oracle import layout
    r, row = int(layout.owner(p, st.N, st.I)), int(layout.local_row(p, st.N, st.I))
    return r, int(st.bt[b][row // st.P]) * st.P + row % st.P


# byte of a cached row: a scale of each CTA's half of the dims, rope dims of each half
PLACES = {"first scale": (256, 0x7F), "last scale": (287, 0xFF), "rope": (288 + 1, 0x7F), "last rope": (288 + 127, 0xFF)}


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("H,q_len", [(16, 1), (17, 1), (128, 1), (96, 3), (5, 2)])
@pytest.mark.parametrize("N,lens,at", [
    (1, [700], [(0, 699)]),                                     # one shard, the newest key
    (1, [9000, 300, 77], [(0, 5), (0, 8990), (2, 40)]),         # units cut by range boundaries
    (4, [3000, 61, 4], [(0, 1001), (1, 0), (2, 1)]),
])
def test_q4_visible_nan(N, lens, at, H, q_len, place):
    from test_gpu_q4 import Q4State
    st = Q4State(lens, H, q_len, N, 1, 64, seed=7 + H, base=1)
    byte, value = PLACES[place]

    def spoil(st):
        for b, p in at:
            r, row = slot_of(st, b, p)
            st.arena[r, row, byte] = value
            if byte >= 288:                                     # a bf16 NaN: exponent bits and a mantissa bit
                st.arena[r, row, byte - 1] = 0xC0

    (o, lse), (o2, lse2) = runs(st, spoil)
    bad = torch.zeros(o.shape[:-1], dtype=torch.bool)
    for b, p in at:
        for t in range(q_len):
            if p <= lens[b] - q_len + t:
                bad[slot_of(st, b, p)[0], b, t] = True
    seen = [(b, p) for b, p in at if p <= lens[b] - q_len]      # by every query token
    for t in range(q_len):                                      # (a key that only later tokens see: see below)
        if len(seen) == len(at):
            compare(o[:, :, t], o2[:, :, t], bad[:, :, t])
            compare(lse[:, :, t], lse2[:, :, t], bad[:, :, t])
        else:
            assert bool(torch.isnan(o2[:, :, t][bad[:, :, t]]).all()) and bool(torch.isnan(lse2[:, :, t][bad[:, :, t]]).all())


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("H,q_len", [(16, 1), (17, 1), (128, 2)])
def test_q4_nan_and_infinite_queries(H, q_len, value):
    """A query row with a NaN, or whose scores are all infinite or NaN, is NaN; the rows beside it are not."""
    from test_gpu_q4 import Q4State
    st = Q4State([4000, 90], H, q_len, 2, 1, 64, seed=3)

    def spoil(st):
        st.q[0, 0, 3, 17] = value
        st.q[1, q_len - 1, H - 1, 575] = value

    (o, lse), (o2, lse2) = runs(st, spoil)
    bad = torch.zeros(o.shape[:-1], dtype=torch.bool)
    bad[:, 0, 0, 3] = bad[:, 1, q_len - 1, H - 1] = True
    compare(o, o2, bad)
    compare(lse, lse2, bad)


@pytest.mark.parametrize("dim", [0, 300, 530, 575])
@pytest.mark.parametrize("name,over", [
    ("tiny", dict(B=3, S=700, H=7)), ("k3", dict(B=2, S=9000)), ("dsv3", dict(B=2, S=5000)), ("ragged", dict(B=3, S=3000, S_min=400)),
])
def test_bf16_visible_nan(name, over, dim):
    """The same in the bf16 cache; a NaN in a query row as well."""
    import workloads
    from harness import GpuState
    from oracle import layout
    st = GpuState(workloads.config(name, **over))
    cfg, d = st.cfg, st.dec
    outs, bad = [], torch.zeros(cfg.N, cfg.B, cfg.q_len, cfg.H, dtype=torch.bool)
    for spoil in (False, True):
        if spoil:
            for b, p in ((0, 5), (1, int(st.S[1]) - cfg.q_len)):       # seen by every query token
                r, row = int(layout.owner(p, cfg.N, cfg.I)), int(layout.local_row(p, cfg.N, cfg.I))
                d.arena[r, int(st.bt[b, row // cfg.P]) * cfg.P + row % cfg.P, dim] = NAN
                bad[r, b] = True
            st.q[cfg.B - 1, 0, 2, dim] = NAN
            bad[:, cfg.B - 1, 0, 2] = True
        o, lse = st.decode()
        outs.append((d.o_part.clone(), d.lse_part.clone(), o.clone(), lse.clone()))
        assert d.status_bits() == 0
    for clean, got, rows in zip(*outs, (bad, bad, bad.any(0), bad.any(0))):
        compare(clean, got, rows)


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("H,q_len", [(8, 2), (1, 16), (5, 3), (6, 3), (9, 7), (128, 4), (16, 64), (96, 5)])
@pytest.mark.parametrize("N,lens", [(1, [700, 64]), (1, [9000, 130, 65]), (4, [3000, 261, 68])])
def test_q4_nan_that_only_later_tokens_see(N, lens, H, q_len, place):
    """Draft tokens' rows hold NaN: the query tokens before them keep their bits, the others are NaN."""
    from test_gpu_q4 import Q4State
    st = Q4State(lens, H, q_len, N, 1, 16, seed=9 + H, base=1)
    byte, value = PLACES[place]
    at = [(b, S - 1 - k) for b, S in enumerate(lens) for k in ((0,), (q_len - 2,), (q_len // 2, 0))[b % 3]]

    def spoil(st):
        for b, p in at:
            r, row = slot_of(st, b, p)
            st.arena[r, row, byte] = value
            if byte >= 288:
                st.arena[r, row, byte - 1] = 0xC0

    (o, lse), (o2, lse2) = runs(st, spoil)
    bad = torch.zeros(o.shape[:-1], dtype=torch.bool)
    for b, p in at:
        for t in range(q_len):
            if p <= lens[b] - q_len + t:
                bad[slot_of(st, b, p)[0], b, t] = True
    assert bool(bad.any()) and not bool(bad.all())
    compare(o, o2, bad)
    compare(lse, lse2, bad)
