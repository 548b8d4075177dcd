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
