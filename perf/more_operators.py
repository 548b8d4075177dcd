"""Norms with rotation into the cache, and eviction by attention weight, as measured cases.

Five kinds of case:

  query    dcp_q_norm_rope: RMS norm of each head's 192 query dims, the last 64 rotated by position
  store    dcp_kv_norm_rope_append (bf16 cache) or dcp_kv_norm_rope_append_q4: RMS norm of the 512 latent dims of a
           projection's rows, their 64 position dims rotated, written into the owners' pools.  With the 4-bit cache
           the rows are read back (dcp_kv_read_q4) as the values the cache stands for
  weigh    dcp_mla_key_weights(_q4): what weight every cached row got from a step's queries, added to what it had
  select   dcp_evict_select: the rows each shard keeps of each request
  compact  dcp_kv_compact(_q4): kept rows, and their weights, moved to the front of their shard in place.  With the
           4-bit cache the rows are read back

The 416-byte rows of the 4-bit cache: 256 bytes of codes, 32 e4m3 scales, 64 bf16 values.  32-bit word k of the codes
holds dims 8k .. 8k + 7: dim 8k + 2i in bits [4i, 4i + 4), dim 8k + 2i + 1 in bits [16 + 4i, 20 + 4i), each as its code
plus 8; the scale of 16 dims is the e4m3 value nearest to their largest magnitude / 7.

`run` computes an operator from elementary torch operations, or with `own` set makes the library's calls.
"""

from __future__ import annotations

import math

import torch

own = False

DK, DV, DR, DQ, GROUP, ROW = 576, 512, 64, 192, 16, 416
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
LOG2E = 1.4426950408889634
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)      # bit of dim 8k + j inside word k
MOST_SCORES = 64 * 96 * 131072              # query rows times keys of the largest weigh case
MOST_QUERY = 8192 * 128                     # query rows of the largest query case
MOST_MOVED = 16 * 32768                     # rows kept in the largest compact case


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the queries of one decode step, 64 requests
        dict(name="query-step", kind="query", T=64, H=96, norm=True, halves=False, far=131072),
        # an 8192-token chunk's queries, far into a long context
        dict(name="query-chunk", kind="query", T=8192, H=128, norm=True, halves=True, far=1040384),
        # one new token for each of 64 requests, on a 4-bit cache
        dict(name="store-step-q4", kind="store", q4=True, B=64, tokens=1, start=8191, N=8, I=1, P=64, held=8, pad=0,
             halves=False, shift=0),
        # an 8192-token chunk of each of 4 requests; after an eviction a token's place is not its rotation's position
        dict(name="store-chunk", kind="store", q4=False, B=4, tokens=8192, start=24576, N=8, I=1, P=64, held=8, pad=0,
             halves=False, shift=4096),
        # one short request of one model-parallel slice: latency alone
        dict(name="weigh-tiny", kind="weigh", q4=False, B=1, H=16, q_len=1, S=1024, S_min=1024, N=4, I=1, P=16, held=4,
             base=0, decay=1.0),
        # a decode step of 64 requests of 128k tokens, 96 heads, base-2 lse
        dict(name="weigh-k3", kind="weigh", q4=False, B=64, H=96, q_len=1, S=131072, S_min=131072, N=8, I=1, P=64,
             held=8, base=1, decay=1.0),
        # the last 64 tokens of two prompts as the window that judges the others
        dict(name="weigh-window", kind="weigh", q4=False, B=2, H=96, q_len=64, S=32768, S_min=32768, N=8, I=1, P=64,
             held=8, base=0, decay=0.0),
        # a decode step of 32 requests of 32k tokens, 128 heads, 4-bit cache
        dict(name="weigh-dsv3-q4", kind="weigh", q4=True, B=32, H=128, q_len=1, S=32768, S_min=32768, N=8, I=1, P=64,
             held=8, base=0, decay=0.9),
        # one request cut by a quarter
        dict(name="select-tiny", kind="select", B=1, S=4096, S_min=4096, new=3001, N=4, I=1, P=16, held=4, sinks=4,
             recent=128),
        # 64 requests of 128k tokens halved
        dict(name="select-k3", kind="select", B=64, S=131072, S_min=131072, new=65536, N=8, I=1, P=64, held=8, sinks=16,
             recent=1024),
        # 16 requests of 64k tokens halved
        dict(name="compact-half", kind="compact", q4=False, B=16, S=65536, S_min=65536, new=32768, N=8, I=1, P=64,
             held=8),
        # a few requests of very different lengths, 4-bit cache, block round-robin
        dict(name="compact-ragged-q4", kind="compact", q4=True, B=5, S=9001, S_min=700, new=2500, N=4, I=4, P=16,
             held=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["query", "store", "weigh", "weigh", "select", "compact"])
    if kind == "query":
        H = _log(rng, 1, 128)
        return dict(kind=kind, T=_log(rng, 1, MOST_QUERY // H // 4), H=H, norm=rng.random() < 0.8,
                    halves=rng.random() < 0.5, far=_log(rng, 1, 1 << 20))
    N = rng.choice([1, 2, 3, 4, 8, 16])
    P = rng.choice([8, 16, 32, 64, 128])
    I = rng.choice([1, 1, 2, 4, 8])
    held = rng.choice([N, N, max(1, N // 2)])
    q4 = rng.random() < 0.4
    if kind == "store":
        B = _log(rng, 1, 128)
        return dict(kind=kind, q4=q4, B=B, tokens=_log(rng, 1, max(2, (1024 if q4 else 32768) // B)),
                    start=_log(rng, 1, 16384), N=N, I=I, P=P, held=held, pad=rng.choice([0, 0, _log(rng, 1, 500)]),
                    halves=rng.random() < 0.5, shift=rng.choice([0, _log(rng, 1, 1 << 19)]))
    if kind == "weigh":
        B, H, q_len = _log(rng, 1, 64), _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 7, 16, 61])
        top = max(600, min(131072, MOST_SCORES // 2 // (B * H * q_len)))
        S = _log(rng, 512, top)
        return dict(kind=kind, q4=q4, B=B, H=H, q_len=q_len, S=S, S_min=max(q_len, rng.choice([S, S, S // 40])), N=N,
                    I=I, P=P, held=held, base=rng.randrange(2), decay=rng.choice([1.0, 0.9, 0.0]))
    if kind == "select":
        B = _log(rng, 1, 64)
        S = _log(rng, 256, 4194304 // B)
        return dict(kind=kind, B=B, S=S, S_min=rng.choice([S, S // 20 + 1]), new=max(1, int(S * rng.uniform(0.1, 0.95))),
                    N=N, I=I, P=P, held=held, sinks=rng.choice([0, 4, 64]), recent=rng.choice([0, 32, S // 16]))
    B = _log(rng, 1, 64)
    S = _log(rng, 256, MOST_MOVED // B)
    return dict(kind=kind, q4=q4, B=B, S=S, S_min=rng.choice([S, S // 20 + 1]), new=max(1, int(S * rng.uniform(0.1, 0.95))),
                N=N, I=I, P=P, held=held)


def _spread(B, lo, hi):
    """B lengths in [lo, hi], spread over their logarithm."""
    if lo >= hi:
        return [hi] * B
    at = [((b + 1) * 0.6180339887498949) % 1.0 for b in range(B)]
    return [min(hi, max(lo, int(math.exp(math.log(lo + 1) + u * (math.log(hi + 1) - math.log(lo + 1)))) - 1)) for u in at]


def _lens(case):
    return _spread(case["B"], case["S_min"], case["S"])


def _new(case):
    """Lengths after an eviction: every request to `new`, or, where it has no more, to all but one of its own."""
    return [min(case["new"], max(0, S - 1)) for S in _lens(case)]


def _share(case, x):
    """Positions in [0, x) of each held shard."""
    N, I = case["N"], case["I"]
    return [(x // (N * I)) * I + min(max(x % (N * I) - r * I, 0), I) for r in range(case["held"])]


def _mine(case, x):
    return sum(_share(case, x))


def work(case):
    if case["kind"] == "query":
        rows = case["T"] * case["H"]
        return {"bytes": rows * DQ * 4 + case["T"] * 8, "flops": rows * (4 * DQ + 3 * DR)}
    if case["kind"] == "store":
        moved = sum(_mine(case, case["start"] + b + case["tokens"]) - _mine(case, case["start"] + b)
                    for b in range(case["B"]))
        back = ROW + DK * 2 if case["q4"] else 0        # rows read back
        return {"bytes": moved * (DK * 2 + (ROW if case["q4"] else DK * 2) + back + 16), "flops": moved * 4 * DK}
    if case["kind"] == "weigh":
        rows = case["B"] * case["q_len"] * case["H"]
        keys = pairs = 0
        for S in _lens(case):
            keys += _mine(case, S)
            pairs += case["H"] * sum(_mine(case, S - case["q_len"] + t + 1) for t in range(case["q_len"]))
        return {"bytes": keys * ((ROW if case["q4"] else DK * 2) + (8 if case["decay"] else 4)) + rows * (DK * 2 + 4),
                "flops": 2 * DK * pairs}
    keys, kept = sum(_mine(case, S) for S in _lens(case)), sum(_mine(case, m) for m in _new(case))
    if case["kind"] == "select":
        return {"bytes": 4 * keys + 4 * kept, "flops": 0}
    width = ROW if case["q4"] else DK * 2
    return {"bytes": kept * (2 * width + 4 + 8 + ((ROW + DK * 2) if case["q4"] else 0)), "flops": 0}


# ---------------------------------------------------------------- inputs
def _quantise(x):
    """[..., 512] -> (codes int32 in [-7, 7], scales f32 that e4m3 holds), in 64 bits next to a border."""
    g = x.double().unflatten(-1, (DV // GROUP, GROUP))
    s = (g.abs().amax(-1, keepdim=True) / 7.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    c = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
    return c.clamp(-7, 7).to(torch.int32).flatten(-2), s.squeeze(-1).float()


def _pack(x):
    """bf16 [..., 576] -> the 416 bytes of its cached row."""
    c, s = _quantise(x[..., :DV])
    sh = torch.tensor(SHIFTS, dtype=torch.int64, device=x.device)
    w = ((c.long() + 8).unflatten(-1, (DV // 8, 8)) << sh).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return torch.cat([w.contiguous().view(torch.uint8), s.to(torch.float8_e4m3fn).view(torch.uint8),
                      x[..., DV:].contiguous().view(torch.uint8)], -1)


def _unpack(row):
    """416 cached bytes [..., 416] -> the f32 values [..., 576] they stand for."""
    sh = torch.tensor(SHIFTS, dtype=torch.int32, device=row.device)
    w = row[..., :DV // 2].contiguous().view(torch.int32).unsqueeze(-1)
    c = (((w >> sh) & 15) - 8).float().flatten(-2)
    s = row[..., DV // 2:DV // 2 + DV // GROUP].contiguous().view(torch.float8_e4m3fn).float()
    c = (c.unflatten(-1, (DV // GROUP, GROUP)) * s.unsqueeze(-1)).flatten(-2)
    return torch.cat([c, row[..., DV // 2 + DV // GROUP:].contiguous().view(torch.bfloat16).float()], -1)


def _table(g, npages, spare, dev):
    """(block table [B, max], pool pages): a shuffled assignment, -1 behind a request's pages."""
    most, total = max(1, max(npages)), sum(npages) + spare
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    n = torch.tensor(npages, device=dev)
    k = torch.arange(most, device=dev)
    at = (torch.cumsum(n, 0) - n)[:, None] + k
    return torch.where(k < n[:, None], perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)), total


def _fill_arena(s, g, dev):
    """Pools of N(0, 1) rows."""
    rows = s["pages"] * s["P"]
    s["arena"] = torch.empty(s["held"], rows, ROW if s["q4"] else DK, dtype=torch.uint8 if s["q4"] else torch.bfloat16,
                             device=dev)
    for r in range(s["held"]):
        for a in range(0, rows, 1 << 20):
            x = torch.randn(min(1 << 20, rows - a), DK, generator=g, device=dev).to(torch.bfloat16)
            s["arena"][r, a:a + (1 << 20)] = _pack(x) if s["q4"] else x


def _merged_lse(s, lens):
    """Each query row's log-sum-exp over what it sees on the held shards, request by request (natural logarithm)."""
    N, I, P = s["N"], s["I"], s["P"]
    out = torch.empty(s["B"], s["q_len"], s["H"], device=s["q"].device)
    for b, S in enumerate(lens):
        p = torch.arange(S, device=s["q"].device)
        own_p = (p // I) % N
        p = p[own_p < s["held"]]
        owner, row = (p // I) % N, p // (N * I) * I + p % I
        x = s["arena"][owner, s["bt"][b, row // P].long() * P + row % P]
        x = (s["q"][b].float().flatten(0, 1) @ (_unpack(x) if s["q4"] else x.float()).T * SCALE).view(s["q_len"], s["H"], -1)
        last = S - s["q_len"] + torch.arange(s["q_len"], device=p.device)
        out[b] = torch.logsumexp(x.masked_fill(p > last[:, None, None], -math.inf), -1)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, DR, 2, device=dev, dtype=torch.float64) / DR)).float()
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if case["kind"] == "query":
        T, H = case["T"], case["H"]
        s["q"] = (2.0 * torch.randn(T, H, DQ, generator=g, device=dev)).to(torch.bfloat16)
        s["pos"] = case["far"] + torch.arange(T, device=dev) if T > 512 else torch.randint(
            0, case["far"], (T,), generator=g, device=dev)
        s["gamma"] = (1.0 + 0.2 * torch.randn(DQ, generator=g, device=dev)).to(torch.bfloat16)
        s["out"] = torch.empty(T, H, DQ, dtype=torch.bfloat16, device=dev)
        return s
    span = case["N"] * case["P"]
    if case["kind"] == "store":
        first = [case["start"] + b for b in range(case["B"])]
        last = [a + case["tokens"] for a in first]
        s["bt"], s["pages"] = _table(g, [-(-x // span) for x in last], 3, dev)
        pos = torch.cat([torch.arange(a, e, device=dev) for a, e in zip(first, last)])
        req = torch.cat([torch.full((e - a,), b, dtype=torch.int32, device=dev)
                         for b, (a, e) in enumerate(zip(first, last))])
        pad = torch.full((case["pad"],), -1, device=dev)
        s["pos"], s["req"] = torch.cat([pos, pad]), torch.cat([req, pad.to(torch.int32)])
        s["rope_pos"] = torch.where(s["pos"] >= 0, s["pos"] + case["shift"], -1)
        # the latent rows are the last 576 columns of a joint projection's output
        s["rows"] = (2.0 * torch.randn(s["pos"].numel(), 1024 + DK, generator=g, device=dev)).to(torch.bfloat16)[:, 1024:]
        s["gamma"] = (1.0 + 0.2 * torch.randn(DV, generator=g, device=dev)).to(torch.bfloat16)
        width, dtype = (ROW, torch.uint8) if case["q4"] else (DK, torch.bfloat16)
        s["arena"] = torch.zeros(case["held"], s["pages"] * case["P"], width, dtype=dtype, device=dev)
        if case["q4"]:
            s["kv"] = torch.zeros(s["pos"].numel(), DK, dtype=torch.bfloat16, device=dev)
        return s
    lens = _lens(case)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int64, device=dev)
    s["bt"], s["pages"] = _table(g, [max(1, -(-x // span)) for x in lens], 0, dev)
    wide = s["bt"].shape[1] * case["P"]
    if case["kind"] == "weigh":
        _fill_arena(s, g, dev)
        rows = (case["B"], case["q_len"], case["H"])
        s["q"] = torch.randn(*rows, DK, generator=g, device=dev).to(torch.bfloat16)
        s["lse"] = _merged_lse(s, lens) * (LOG2E if case["base"] else 1.0)
        s["old_lens"] = s["seq_lens"] - case["q_len"]
        # what some ten earlier steps left
        s["weights"] = torch.rand(case["held"], case["B"], wide, generator=g, device=dev) * (
            20.0 * case["H"] * case["q_len"] / case["S"])
        return s
    s["new_lens"] = torch.tensor(_new(case), dtype=torch.int64, device=dev)
    # accumulated weights: a few rows have most of them, some none at all, and small ones are often alike
    w = torch.exp(2.0 * torch.randn(case["held"], case["B"], wide, generator=g, device=dev))
    s["weights"] = torch.where(w < 0.05, torch.zeros_like(w), torch.where(w < 0.3, (w * 4096).round() / 4096, w))
    keep = max(1, max(max(_share(case, m)) for m in _new(case)))
    s["kept"] = torch.full((case["held"], case["B"], keep), -1, dtype=torch.int32, device=dev)
    if case["kind"] == "compact":
        _fill_arena(s, g, dev)
        # rows kept: a random ascending choice of count(new) of count(length) rows, for each shard and request
        n = torch.tensor([_share(case, x) for x in lens], device=dev).T[:, :, None]
        m = torch.tensor([_share(case, x) for x in _new(case)], device=dev).T[:, :, None]
        x = torch.rand(case["held"], case["B"], wide, generator=g, device=dev)
        x = torch.where(torch.arange(wide, device=dev) < n, x, 2.0)
        order = torch.argsort(x, -1)[..., :keep]
        order = torch.where(torch.arange(keep, device=dev) < m, order, wide).sort(-1).values
        s["kept"].copy_(torch.where(torch.arange(keep, device=dev) < m, order, -1))
        if case["q4"]:                                  # tokens whose rows are read back: what every request has left
            left = _new(case)
            s["pos"] = torch.cat([torch.arange(x, device=dev) for x in left])
            s["req"] = torch.cat([torch.full((x,), b, dtype=torch.int32, device=dev) for b, x in enumerate(left)])
            s["kv"] = torch.zeros(s["pos"].numel(), DK, dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- plain forms
def _place(s, pos, req):
    """(owner, slot) of tokens; slot -1 where there is no token."""
    N, I, P = s["N"], s["I"], s["P"]
    owner = torch.where(pos >= 0, (pos // I) % N, -1)
    row = torch.where(pos >= 0, (pos // (N * I)) * I + pos % I, -1)
    page = s["bt"][req.clamp(min=0).long(), (row.clamp(min=0)) // P].long()
    return owner, torch.where(pos >= 0, page * P + row % P, -1)


def _norm(x, gamma):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()


def _rotate(x, pos, inv_freq, halves):
    """[T, ..., 64] rotated by its positions: pairs (i, i + 32), or (2i, 2i + 1)."""
    a = pos.double()[:, None] * inv_freq.double()                                     # angles of far positions: 64 bits
    a = a.view(a.shape[0], *([1] * (x.dim() - 2)), DR // 2)
    c, d = torch.cos(a).float(), torch.sin(a).float()
    u, v = (x[..., :DR // 2], x[..., DR // 2:]) if halves else (x[..., 0::2], x[..., 1::2])
    u, v = u * c - v * d, u * d + v * c
    return torch.cat([u, v], -1) if halves else torch.stack([u, v], -1).flatten(-2)


def _query_plain(s):
    x = s["q"].float()
    if s["norm"]:
        x = _norm(x, s["gamma"])
    y = _rotate(x[..., DQ - DR:], s["pos"], s["inv_freq"], s["halves"])
    s["out"].copy_(torch.cat([x[..., :DQ - DR], y], -1))
    return {"q": s["out"]}


def _read_plain(s, width):
    """The read-back of a 4-bit cache's tokens (rows of other shards as they were)."""
    owner, slot = _place(s, s["pos"], s["req"])
    mine = (owner >= 0) & (owner < s["held"])
    at = torch.where(mine, owner * s["arena"].shape[1] + slot, 0)
    s["kv"].copy_(torch.where(mine[:, None], _unpack(s["arena"].view(-1, width)[at]).to(torch.bfloat16), s["kv"]))


def _store_plain(s):
    x = s["rows"].float()
    y = _rotate(x[:, DV:], s["rope_pos"], s["inv_freq"], s["halves"])
    x = torch.cat([_norm(x[:, :DV], s["gamma"]), y], -1).to(torch.bfloat16)
    owner, slot = _place(s, s["pos"], s["req"])
    mine = (owner >= 0) & (owner < s["held"])
    flat = s["arena"].view(-1, s["arena"].shape[-1])
    at = torch.where(mine, owner * s["arena"].shape[1] + slot, 0)
    first = torch.argmax(mine.to(torch.int32))                                        # entries that are not held
    data = torch.where(mine[:, None], _pack(x) if s["q4"] else x, flat[at])           # repeat the first held one
    flat[torch.where(mine, at, at[first])] = torch.where(mine[:, None], data, data[first])
    if s["q4"]:
        _read_plain(s, ROW)
        return {"kv": s["kv"]}
    return {"arena": s["arena"]}


def _weigh_plain(s):
    N, I, P, n, B, q_len, H = (s[k] for k in ("N", "I", "P", "held", "B", "q_len", "H"))
    dev = s["q"].device
    k = torch.arange(s["weights"].shape[2], device=dev)
    slot = s["bt"].clamp(min=0).long()[:, k // P] * P + k % P                         # [B, L]
    kv = _unpack(s["arena"][:, slot]) if s["q4"] else s["arena"][:, slot].float()     # [n, B, L, 576]
    x = torch.matmul(kv, s["q"].float().view(B, q_len * H, DK).transpose(-1, -2))     # [n, B, L, R]
    lse = (s["lse"] / LOG2E if s["base"] else s["lse"]).view(B, 1, q_len * H)
    x = torch.exp(x * SCALE - lse)
    at = (k // I * N + torch.arange(n, device=dev)[:, None]) * I + k % I              # [n, L] positions
    last = (s["seq_lens"][:, None] - q_len + torch.arange(q_len, device=dev)).repeat_interleave(H, 1)
    x = torch.where(at[:, None, :, None] <= last[:, None, :], x, 0.0).sum(-1)         # [n, B, L]
    old = torch.where(at[:, None, :] < s["old_lens"][:, None], s["decay"] * s["weights"], 0.0)
    live = at[:, None, :] < s["seq_lens"][:, None]
    s["weights"].copy_(torch.where(live, old + x, s["weights"]))
    return {"weights": s["weights"]}


def _count(s, x):
    """Rows of each held shard below position x [B] -> [held, B]."""
    N, I = s["N"], s["I"]
    r = torch.arange(s["held"], device=x.device)[:, None]
    return x // (N * I) * I + (x % (N * I) - r * I).clamp(min=0, max=I)


def _select_plain(s):
    n, m = _count(s, s["seq_lens"]), _count(s, s["new_lens"])
    a = _count(s, s["seq_lens"].clamp(max=s["sinks"]))                                # rows below a: sinks
    z = torch.maximum(a, _count(s, (s["seq_lens"] - s["recent"]).clamp(min=0)))       # rows from z on: recent
    ns = torch.minimum(a, m)
    nr = torch.minimum(m - ns, n - z)
    row = torch.arange(s["weights"].shape[2], device=n.device)
    mid = (row >= a[..., None]) & (row < z[..., None])
    order = torch.sort(torch.where(mid, s["weights"], -1.0), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, row.expand_as(order).contiguous())
    keep = (row < ns[..., None]) | ((row >= (n - nr)[..., None]) & (row < n[..., None])) | (
        mid & (rank < (m - ns - nr)[..., None]))
    size = s["kept"].shape[2]
    at = torch.where(keep, torch.cumsum(keep.long(), -1) - 1, size)                   # one place for what is dropped
    out = torch.cat([s["kept"], s["kept"][..., :1]], -1)
    s["kept"].copy_(out.scatter_(-1, at, row.to(torch.int32).expand_as(at).contiguous())[..., :size])
    return {"kept": s["kept"]}


def _compact_plain(s):
    P, n, B = s["P"], s["held"], s["B"]
    i = torch.arange(s["kept"].shape[2], device=s["kept"].device)
    live = i < _count(s, s["new_lens"])[..., None]                                    # [n, B, K]
    src = torch.where(live, s["kept"].long(), 0)
    b = torch.arange(B, device=i.device)[:, None]
    pool = (torch.arange(n, device=i.device) * s["arena"].shape[1])[:, None, None]
    frm = (pool + s["bt"].clamp(min=0).long()[b, src // P] * P + src % P).flatten()
    to = (pool + (s["bt"].clamp(min=0).long()[b, i // P] * P + i % P)).flatten()
    flat, ok = s["arena"].view(-1, s["arena"].shape[-1]), live.flatten()
    first = torch.argmax(ok.to(torch.int32))                                          # entries behind a unit's last
    flat[torch.where(ok, to, to[first])] = flat[torch.where(ok, frm, frm[first])]     # repeat the first live one
    w = torch.gather(s["weights"], -1, src)
    s["weights"][..., :i.numel()] = torch.where(live, w, s["weights"][..., :i.numel()])
    if s["q4"]:
        _read_plain(s, ROW)
        return {"kv": s["kv"], "weights": s["weights"]}
    return {"arena": s["arena"], "weights": s["weights"]}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    import context_sharded_mla_gb300 as dcp

    style = dcp.DCP_ROPE_HALVES if s.get("halves") else dcp.DCP_ROPE_PAIRS
    if s["kind"] == "query":
        dcp.dcp_q_norm_rope(s["q"], s["pos"], s["out"], gamma=s["gamma"] if s["norm"] else None, eps=EPS,
                            inv_freq=s["inv_freq"], rope_style=style, status=s["status"])
        return {"q": s["out"]}
    lay = dcp.Layout(s["N"], s["I"], s["P"])
    bt, wide = s["bt"], s["bt"].shape[1]
    if s["kind"] == "store":
        store = dcp.dcp_kv_norm_rope_append_q4 if s["q4"] else dcp.dcp_kv_norm_rope_append
        store(lay, 0, s["held"], s["rows"], s["pos"], s["req"], bt, wide, s["arena"], s["pages"], s["status"],
              gamma=s["gamma"], eps=EPS, inv_freq=s["inv_freq"], rope_style=style, rope_pos=s["rope_pos"])
    elif s["kind"] == "weigh":
        weigh = dcp.dcp_mla_key_weights_q4 if s["q4"] else dcp.dcp_mla_key_weights
        weigh(lay, 0, s["held"], s["q"], s["arena"], s["pages"], bt, wide, s["seq_lens"], SCALE,
              dcp.DCP_LSE_BASE_2 if s["base"] else dcp.DCP_LSE_BASE_E, s["lse"], s["weights"], s["status"],
              old_lens=s["old_lens"], decay=s["decay"])
        return {"weights": s["weights"]}
    elif s["kind"] == "select":
        dcp.dcp_evict_select(lay, 0, s["held"], s["seq_lens"], s["new_lens"], s["sinks"], s["recent"], s["weights"],
                             s["kept"], s["status"])
        return {"kept": s["kept"]}
    else:
        compact = dcp.dcp_kv_compact_q4 if s["q4"] else dcp.dcp_kv_compact
        compact(lay, 0, s["held"], s["kept"], s["new_lens"], bt, wide, s["arena"], s["pages"], s["status"],
                weights=s["weights"])
    if not s["q4"]:
        return {"arena": s["arena"]} if s["kind"] == "store" else {"arena": s["arena"], "weights": s["weights"]}
    dcp.dcp_kv_read_q4(lay, 0, s["held"], s["arena"], s["pages"], s["pos"], s["req"], bt, wide, s["kv"], s["status"])
    return {"kv": s["kv"]} if s["kind"] == "store" else {"kv": s["kv"], "weights": s["weights"]}


def run(state):
    if own:
        return _own(state)
    return {"query": _query_plain, "store": _store_plain, "weigh": _weigh_plain, "select": _select_plain,
            "compact": _compact_plain}[state["kind"]](state)


# ---------------------------------------------------------------- in 64 bits
def _exact_rows(raw):
    """The values cached rows stand for, in 64 bits, byte by byte."""
    raw = raw.long()
    d = torch.arange(DV, device=raw.device)
    j = d % 8
    bit = 4 * (j // 2) + 16 * (j % 2)
    code = ((raw[..., 4 * (d // 8) + bit // 8] >> (bit % 8)) & 15) - 8
    e = raw[..., DV // 2 + d // GROUP]
    power, frac = (e >> 3) & 15, (e & 7).double()
    size = torch.where(power > 0, (1 + frac / 8) * torch.exp2((power - 7).double()), frac / 512)
    out = torch.empty(*raw.shape[:-1], DK, dtype=torch.float64, device=raw.device)
    out[..., :DV] = code.double() * size
    tail = raw[..., DV // 2 + DV // GROUP:].unflatten(-1, (DK - DV, 2))
    bits = (tail[..., 0] + 256 * tail[..., 1]) << 16
    out[..., DV:] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).view(torch.float32).double()
    return out


def _exact_values(x):
    """What the cache holds of rows, in 64 bits: the scale by search among all e4m3 values, codes by comparison."""
    x = x.double()
    e = torch.arange(127, device=x.device)
    table = torch.where(e >= 8, (1 + (e % 8).double() / 8) * torch.exp2((e // 8 - 7).double()), e.double() / 512)
    out = x.clone()
    for g in range(DV // GROUP):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        want = part.abs().amax(1) / 7
        up = torch.searchsorted(table, want).clamp(max=126)
        down = (up - 1).clamp(min=0)
        a, b = want - table[down], table[up] - want
        pick = torch.where((a < b) | ((a == b) & (down % 2 == 0)), down, up)
        size = table[pick][:, None]
        low = torch.floor(part / torch.where(size > 0, size, torch.ones_like(size)))
        a, b = part - low * size, (low + 1) * size - part
        code = torch.where((a < b) | ((a == b) & (low % 2 == 0)), low, low + 1)
        out[:, g * GROUP:(g + 1) * GROUP] = torch.where(size > 0, code.clamp(-7, 7) * size, torch.zeros_like(part))
    return out


def _exact_turn(x, pos, inv_freq, halves):
    """64 dims as 32 complex numbers times exp(i angle)."""
    j = torch.arange(DR // 2, device=x.device)
    re, im = (j, j + DR // 2) if halves else (2 * j, 2 * j + 1)
    angle = pos.double()[:, None] * inv_freq.double()
    z = torch.complex(x[..., re], x[..., im])
    z = z * torch.polar(torch.ones_like(angle), angle).view(angle.shape[0], *([1] * (x.dim() - 2)), DR // 2)
    out = torch.empty_like(x)
    out[..., re], out[..., im] = z.real, z.imag
    return out


def _exact_scaled(x, gamma):
    size = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS)
    return gamma.double() * x / size


def _exact_moved(case, s):
    """Rows and weights moved, a shard and a request at a time; the 4-bit rows as values, position by position."""
    N, I, P = case["N"], case["I"], case["P"]
    rows = s["arena"] if case["q4"] else s["arena"].double()
    before, weights, values = s["arena"], s["weights"].double(), []
    for b, left in enumerate(_new(case)):
        kv = torch.zeros(left, DK, dtype=torch.float64, device=weights.device)
        for r in range(case["held"]):
            i = torch.arange(_share(case, left)[r], device=weights.device)
            k = s["kept"][r, b, :i.numel()].long()
            moved = before[r, s["bt"][b, k // P].long() * P + k % P]
            weights[r, b, i] = s["weights"][r, b, k].double()
            if case["q4"]:
                kv[(i // I * N + r) * I + i % I] = _exact_rows(moved)
            else:
                rows[r, s["bt"][b, i // P].long() * P + i % P] = moved.double()
        values.append(kv)
    return {"kv": torch.cat(values), "weights": weights} if case["q4"] else {"arena": rows, "weights": weights}


def exact(case, seed):
    if case["kind"] == "select":
        return None                                     # whole numbers
    s = prepare(case, seed)
    if case["kind"] == "compact":
        return _exact_moved(case, s)
    if case["kind"] == "query":
        x = s["q"].double()
        if case["norm"]:
            x = _exact_scaled(x, s["gamma"])
        x[..., DQ - DR:] = _exact_turn(x[..., DQ - DR:].clone(), s["pos"], s["inv_freq"], case["halves"])
        return {"q": x}
    N, I, P = case["N"], case["I"], case["P"]
    if case["kind"] == "store":
        x = s["rows"].double()
        x = torch.cat([_exact_scaled(x[:, :DV], s["gamma"]),
                       _exact_turn(x[:, DV:].clone(), s["rope_pos"], s["inv_freq"], case["halves"])], -1)
        owner = torch.where(s["pos"] >= 0, s["pos"] // I % N, N)
        mine = torch.nonzero(owner < case["held"]).flatten()
        if case["q4"]:
            out = torch.zeros_like(x)
            out[mine] = _exact_values(x[mine].to(torch.bfloat16))     # the cache's input is bf16
            out[mine, DV:] = x[mine, DV:]
            return {"kv": out}
        out = torch.zeros(s["arena"].shape, dtype=torch.float64, device=x.device)
        p = s["pos"][mine]
        row = p // (N * I) * I + p % I
        out[owner[mine], s["bt"][s["req"][mine].long(), row // P].long() * P + row % P] = x[mine]
        return {"arena": out}
    out = s["weights"].double()
    for b, S in enumerate(_lens(case)):
        p = torch.arange(S, device=out.device)
        z = s["lse"][b].double() * (math.log(2.0) if case["base"] else 1.0)
        for r in range(case["held"]):
            at = p[(p // I) % N == r]
            if not at.numel():
                continue
            row = at // (N * I) * I + at % I
            kv = s["arena"][r, s["bt"][b, row // P].long() * P + row % P]
            kv = _exact_rows(kv) if case["q4"] else kv.double()
            x = torch.exp((s["q"][b].double().flatten(0, 1) @ kv.T / math.sqrt(192.0)).view(case["q_len"], case["H"], -1)
                          - z[..., None])
            seen = at[None, :] <= S - case["q_len"] + torch.arange(case["q_len"], device=at.device)[:, None]
            got = (x.sum(1) * seen).sum(0)
            keep = torch.where(at < S - case["q_len"], case["decay"] * out[r, b, row], torch.zeros_like(got))
            out[r, b, row] = keep + got
    return {"weights": out}
