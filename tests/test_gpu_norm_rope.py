"""Norm and rotation of queries and latent rows on the GPU, against fp64.

Bounds (u = 2^-24).  A normed value x r g: the squares' sum has at most 30 roundings, r = rsqrt(..) 4 u, two products:
below 2^-18 of itself.  A rotated one: products of such values with a sine and a cosine that are off by 2^-20 (their
arguments' roundings, 2 pi u + pi u, and the hardware functions' 2^-21 in [-pi, pi]), two roundings: 2^-18 + 2^-20 + 2 u,
below 2^-17 (|a| + |b|).  Then one rounding to
bf16, half a step: 2^-8 of the value."""

import numpy as np
import pytest
import torch

from oracle import cache_q4, layout as olayout, norm_rope

from harness import bits, to_f64
from test_gpu_q4 import make_tables

pytestmark = pytest.mark.gpu

FREQ = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float()


def _dcp():
    import context_sharded_mla_gb300 as dcp
    return dcp


def expected(x, gamma, eps, pos, freq, halves, rope_at):
    """(values, bound) of rows x [T, ..., width] whose last 64 dims rotate; gamma over the first rope_at dims or all."""
    y = x.copy()
    if gamma is not None:
        w = len(gamma)
        y[..., :w] = norm_rope.rms_norm(x[..., :w], gamma, eps)
    slack = 2.0 ** -18 * np.abs(y)
    if freq is not None:
        part = y[..., rope_at:]
        size = np.abs(part)
        i = np.arange(64)
        other = (i + 32) % 64 if halves else i ^ 1
        slack[..., rope_at:] = 2.0 ** -17 * (size + size[..., other])
        y[..., rope_at:] = norm_rope.rotate(part, pos, freq, halves)
    if gamma is None:
        slack[..., :rope_at] = 0
        if freq is None:
            slack[:] = 0
    return y, slack + 2.0 ** -8 * (np.abs(y) + slack)


def check(got, want, bound, what):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)) and np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-30)).max()))


@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (2, 96), (64, 96), (301, 128), (5000, 7)])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("norm,rope", [(torch.bfloat16, True), (torch.float32, True), (None, True), (torch.bfloat16, False),
                                       (torch.float32, False), (None, False)])
def test_query(T, H, halves, norm, rope):
    dcp = _dcp()
    g = torch.Generator().manual_seed(T * 131 + H)
    q = (3 * torch.randn(T, H, 192, generator=g)).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = (1 << 24) - 1, 1 << 31
    gamma = (1 + 0.3 * torch.randn(192, generator=g)).to(norm or torch.float32)
    out = torch.full_like(q, 9.0).cuda()
    dcp.dcp_q_norm_rope(q.cuda(), pos.cuda(), out, gamma=gamma.cuda() if norm else None, eps=1e-5,
                        inv_freq=FREQ.cuda() if rope else None, rope_style=int(halves))
    want, bound = expected(to_f64(q), to_f64(gamma) if norm else None, 1e-5, pos.numpy(), FREQ.double().numpy() if rope else None,
                           halves, 128)
    check(to_f64(out), want, bound, "q")


def test_query_views_padding_in_place_and_streams():
    dcp = _dcp()
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(9, 6, 256, generator=g).to(torch.bfloat16).cuda()
    pos = torch.tensor([4, -1, 7, 0, -1, 100000, 3, 2, 1], device="cuda")
    args = dict(gamma=torch.ones(192, device="cuda"), inv_freq=FREQ.cuda())
    out = torch.full((9, 6, 192), 9.0, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_q_norm_rope(wide[..., 32:224], pos, out, **args)                 # rows 256 apart, 64 bytes in
    assert torch.all(out[[1, 4]] == 9.0)                                     # padding: as it was
    same = wide[..., 32:224].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dcp.dcp_q_norm_rope(same, pos, same, stream=side, **args)                # in place, on another stream
    side.synchronize()
    live = pos >= 0
    assert torch.equal(same[live], out[live]) and torch.equal(same[~live], wide[..., 32:224][~live])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([4, -2, 7, 0, -1, 5, 3, 2, 1], device="cuda")
    out.fill_(9.0)
    dcp.dcp_q_norm_rope(wide[..., 32:224], bad, out, status=status, **args)
    assert int(status.item()) == 1 and torch.all(out[[1, 4]] == 9.0)
    dcp.dcp_q_norm_rope(wide[:0, :, 32:224], pos[:0], out[:0], **args)       # no tokens
    with pytest.raises(ValueError):
        dcp.dcp_q_norm_rope(wide[..., 32:224], pos[:3], out, **args)
    with pytest.raises(ValueError):
        dcp.dcp_q_norm_rope(wide[..., 32:224], pos, out, inv_freq=FREQ.double().cuda())
    with pytest.raises(ValueError):
        dcp.dcp_q_norm_rope(wide.transpose(0, 1)[..., 32:224], pos[:6], out, **args)   # rows not equally strided


def run_append(q4, x, pos, req, bt, pool, N, I, P, begin, end, fill=None, **kw):
    dcp = _dcp()
    n = end - begin
    if q4:
        arena = torch.zeros(n, pool * P, 416, dtype=torch.uint8, device="cuda")
    else:
        arena = torch.full((n, pool * P, 576), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = dcp.dcp_kv_norm_rope_append_q4 if q4 else dcp.dcp_kv_norm_rope_append
    fn(dcp.Layout(N, I, P), begin, end, x, pos, req, bt, bt.shape[1], arena, pool, status, **kw)
    return arena, int(status.item())


@pytest.mark.parametrize("N,I,P,begin,end", [(4, 1, 16, 0, 4), (8, 1, 64, 2, 5), (3, 8, 8, 0, 3), (1, 1, 1, 0, 1)])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("norm,rope,shift", [(True, True, 0), (True, True, 777777), (False, True, 3), (True, False, 0),
                                             (False, False, 0)])
def test_append(N, I, P, begin, end, halves, norm, rope, shift):
    dcp = _dcp()
    lens = [1, 37, min(3 * N * P + 5, 700)]
    bt, pool = make_tables(lens, N, P, 2, 7)
    pos = np.concatenate([np.arange(n) for n in lens] + [[-1, -1]]).astype(np.int64)
    req = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[-1, -1]]).astype(np.int32)
    order = np.random.default_rng(1).permutation(len(pos))
    pos, req = pos[order], req[order]
    g = torch.Generator().manual_seed(3)
    x = (2 * torch.randn(len(pos), 704, generator=g)).to(torch.bfloat16)[:, 128:]
    gamma = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.float32 if halves else torch.bfloat16)
    rp = np.where(pos >= 0, pos + shift, -1)
    kw = dict(gamma=gamma.cuda() if norm else None, inv_freq=FREQ.cuda() if rope else None, rope_style=int(halves), eps=1e-6,
              rope_pos=torch.from_numpy(rp).cuda() if shift else None)
    args = (torch.from_numpy(pos).cuda(), torch.from_numpy(req).cuda(), torch.from_numpy(bt).cuda(), pool, N, I, P, begin, end)
    xc = x.cuda() if not x.is_contiguous() else x.clone().cuda()
    wide = torch.zeros(len(pos), 704, dtype=torch.bfloat16, device="cuda")
    wide[:, 128:] = xc
    arena, status = run_append(False, wide[:, 128:], *args, **kw)
    assert status == 0
    want, bound = expected(to_f64(x), to_f64(gamma) if norm else None, 1e-6, rp, FREQ.double().numpy() if rope else None, halves, 512)
    got = to_f64(arena)
    touched = np.zeros(got.shape[:2], bool)
    for t, (p, b) in enumerate(zip(pos, req)):
        if p >= 0 and begin <= olayout.owner(p, N, I) < end:
            row = olayout.local_row(p, N, I)
            at = (int(olayout.owner(p, N, I)) - begin, int(bt[b, row // P] * P + row % P))
            check(got[at], want[t], bound[t], (p, b))
            touched[at] = True
    assert np.all(got[~touched] == 9.0)
    # the 4-bit append is the bf16 one and the quantiser, bit for bit
    arena4, status = run_append(True, wide[:, 128:], *args, **kw)
    assert status == 0
    rows = arena.cpu()[torch.from_numpy(touched)]
    codes, scales = cache_q4.quantise(to_f64(rows)[:, :512])
    packed = cache_q4.pack(codes, scales, bits(rows[:, 512:]))
    got4 = arena4.cpu().numpy()
    assert np.array_equal(got4[touched], packed) and not got4[~touched].any()


@pytest.mark.parametrize("q4", [False, True])
def test_append_of_bad_tokens(q4):
    N, I, P = 2, 1, 8
    bt = torch.tensor([[0, 3], [1, 99]], dtype=torch.int32, device="cuda")
    x = torch.randn(7, 576, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([0, -5, 3, 40, 16, 16, -1], device="cuda")
    req = torch.tensor([0, 0, 9, 0, 1, 0, -1], dtype=torch.int32, device="cuda")
    arena, status = run_append(q4, x, pos, req, bt, 4, N, I, P, 0, 2, gamma=torch.ones(512, device="cuda"), inv_freq=FREQ.cuda())
    assert status == 1 | 2 | 4 | 8
    fill = torch.zeros_like(arena) if q4 else torch.full_like(arena, 9.0)
    rows = (arena != fill).any(-1).nonzero().tolist()
    assert rows == [[0, 0], [0, 24]]                 # token 0 of request 0 and its token 16 (row 8, page 3)


def test_a_nan_stays_in_its_row():
    x = torch.randn(3, 576, device="cuda").to(torch.bfloat16)
    x[1, 7] = float("nan")
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    arena, _ = run_append(False, x, torch.arange(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), bt, 1, 1, 1, 8,
                          0, 1, gamma=torch.ones(512, device="cuda"), inv_freq=FREQ.cuda())
    bad = torch.isnan(arena[0])
    assert bad[1, :512].all() and not bad[1, 512:].any() and not bad[[0, 2]].any()
