"""The 4-bit latent cache and the GPU-built block tables, as measured cases.

Four kinds of case, one per operator (or pair of operators that a program runs together):

  decode    dcp_mla_decode_partial_q4: per-shard partial attention over a latent cache held in 4 bits
  append    dcp_kv_append_q4 and dcp_kv_read_q4: new latent rows quantised into the shards' pools, then
            read back as the values the cache stands for
  relayout  dcp_kv_relayout_q4 and dcp_kv_read_q4: rows of a bf16 prefill pool quantised into the pools,
            then read back
  tables    dcp_block_tables: block tables, free list, positions and slots of a step from request lengths

A cached row is 416 bytes: 256 bytes of codes, 32 scales, 64 bf16 values.  Dims [0, 512) are signed 4-bit
codes with one e4m3 scale for 16 dims; dims [512, 576) are bf16.  32-bit word k of the codes holds dims
8k .. 8k + 7: dim 8k + 2i in bits [4i, 4i + 4), dim 8k + 2i + 1 in bits [16 + 4i, 20 + 4i), each as its
code plus 8.

`run` computes an operator from elementary torch operations, or with `own` set makes the library's calls.
"""

from __future__ import annotations

import math

import torch

own = False

DK, DV, GROUP, ROW = 576, 512, 16, 416
SCALE = 1.0 / math.sqrt(192.0)
LOG2E = 1.4426950408889634
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)      # bit of dim 8k + j inside word k
MOST_SCORES = 64 * 96 * 131072              # rows times keys of the largest decode case


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short request of one model-parallel slice: latency alone
        dict(name="decode-tiny", kind="decode", B=1, H=16, q_len=1, S=1024, S_min=1024, N=4, I=1, P=16, held=4, base=0),
        # a decode step of 32 requests of 32k tokens, 128 heads
        dict(name="decode-dsv3", kind="decode", B=32, H=128, q_len=1, S=32768, S_min=32768, N=8, I=1, P=64, held=8,
             base=0),
        # a decode step of 64 requests of 128k tokens, 96 heads, base-2 lse
        dict(name="decode-k3", kind="decode", B=64, H=96, q_len=1, S=131072, S_min=131072, N=8, I=1, P=64, held=8,
             base=1),
        # a speculative verify of 4 tokens over requests of very different lengths, block round-robin
        dict(name="decode-ragged", kind="decode", B=16, H=128, q_len=4, S=65521, S_min=1021, N=16, I=16, P=64,
             held=16, base=0),
        # a chunk of 64 query tokens over a long prefix (chunked extend)
        dict(name="decode-extend", kind="decode", B=2, H=96, q_len=64, S=32768, S_min=32768, N=8, I=1, P=64, held=8,
             base=0),
        # one new token for each of 64 requests
        dict(name="append-step", kind="append", B=64, tokens=1, start=8191, N=8, I=1, P=64, held=8, pad=0),
        # an 8192-token chunk of each of 4 requests
        dict(name="append-chunk", kind="append", B=4, tokens=8192, start=24576, N=8, I=1, P=64, held=8, pad=0),
        # a padded batch on one rank of a two-rank group: half of the shards, entries behind the last token
        dict(name="append-padded", kind="append", B=37, tokens=29, start=777, N=4, I=2, P=16, held=2, pad=111),
        # two requests of 128k tokens prefilled elsewhere, moved into the shards
        dict(name="relayout-long", kind="relayout", B=2, S=131072, Ps=64, N=8, I=1, P=64, held=8),
        # a short one with an odd length and another page size, block round-robin
        dict(name="relayout-odd", kind="relayout", B=3, S=1237, Ps=48, N=4, I=4, P=16, held=4),
        # a verify step: 4 draft tokens of each of 128 requests placed, then rejected
        dict(name="tables-step", kind="tables", B=128, S=32768, S_min=1024, grow=4, N=8, I=1, P=64),
        # 64 prompts of up to 32k tokens admitted, then released
        dict(name="tables-admit", kind="tables", B=64, S=0, S_min=0, grow=32768, N=8, I=1, P=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "append", "relayout", "tables"])
    N = rng.choice([1, 2, 3, 4, 8, 16])
    P = rng.choice([8, 16, 32, 64, 128])
    I = rng.choice([1, 1, 2, 4, 8])
    held = rng.choice([N, N, max(1, N // 2)])
    if kind == "decode":
        B, H, q_len = _log(rng, 1, 64), _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 7, 16])
        top = max(2048, min(131072, MOST_SCORES // (B * H * q_len)))
        S = _log(rng, 512, top)
        return dict(kind=kind, B=B, H=H, q_len=q_len, S=S, S_min=max(q_len, rng.choice([S, S, S // 40])), N=N, I=I, P=P,
                    held=held, base=rng.randrange(2))
    if kind == "append":
        B = _log(rng, 1, 128)
        return dict(kind=kind, B=B, tokens=_log(rng, 1, max(2, 32768 // B)), start=_log(rng, 1, 16384), N=N, I=I, P=P,
                    held=held, pad=rng.choice([0, 0, _log(rng, 1, 500)]))
    if kind == "relayout":
        B = _log(rng, 1, 16)
        return dict(kind=kind, B=B, S=_log(rng, 16, 262144 // B), Ps=rng.choice([16, 48, 64, 128]), N=N, I=I, P=P,
                    held=held)
    B = _log(rng, 1, 256)
    S = rng.choice([0, _log(rng, 64, 65536)])
    return dict(kind=kind, B=B, S=S, S_min=S // 16, grow=rng.choice([1, 2, 5, _log(rng, 8, 2097152 // B)]), N=N, I=I,
                P=P)


def _spread(B, lo, hi):
    """B lengths in [lo, hi], spread over their logarithm."""
    if lo >= hi:
        return [hi] * B
    at = [((b + 1) * 0.6180339887498949) % 1.0 for b in range(B)]
    return [min(hi, max(lo, int(math.exp(math.log(lo + 1) + u * (math.log(hi + 1) - math.log(lo + 1)))) - 1)) for u in at]


def _lens(case):
    return _spread(case["B"], case["S_min"], case["S"])


def _grown(case):
    """The lengths a tables case grows to: every request by `grow`, or prompts up to `grow` tokens."""
    old = _lens(case)
    if case["grow"] <= 16:
        return [a + case["grow"] for a in old]
    return [a + g for a, g in zip(old, _spread(case["B"], max(1, case["grow"] // 32), case["grow"]))]


def _mine(case, x):
    """Positions in [0, x) of the held shards [0, held)."""
    return sum((x // (case["N"] * case["I"])) * case["I"] + min(max(x % (case["N"] * case["I"]) - r * case["I"], 0), case["I"])
               for r in range(case["held"]))


def work(case):
    if case["kind"] == "decode":
        rows = case["B"] * case["q_len"] * case["H"]
        keys = pairs = 0
        for S in _lens(case):
            keys += _mine(case, S)
            pairs += case["H"] * sum(_mine(case, S - case["q_len"] + t + 1) for t in range(case["q_len"]))
        return {"bytes": keys * ROW + rows * DK * 2 + case["held"] * rows * (DV * 2 + 4), "flops": 2 * (DK + DV) * pairs}
    if case["kind"] in ("append", "relayout"):
        if case["kind"] == "append":
            moved = sum(_mine(case, case["start"] + b + case["tokens"]) - _mine(case, case["start"] + b)
                        for b in range(case["B"]))
        else:
            moved = sum(_mine(case, case["S"] - b) for b in range(case["B"]))
        return {"bytes": moved * 2 * (DK * 2 + ROW), "flops": 4 * moved * DV}
    old, new = _lens(case), _grown(case)
    pages = sum(-(-n // (case["N"] * case["P"])) - -(-a // (case["N"] * case["P"])) for a, n in zip(old, new))
    tokens = sum(new) - sum(old)
    return {"bytes": tokens * (8 + 4 + 4 + 8 + 8) + 16 * pages + case["B"] * 3 * 8, "flops": 0}


# ---------------------------------------------------------------- inputs
def _quantise(x):
    """bf16 [..., 512] -> (codes int32 in [-7, 7], scales f32 that e4m3 holds): the nearest code (ties to even) of
    x over its group's scale, the scale the nearest e4m3 value (at most 448) to the group's largest magnitude / 7."""
    g = x.double().unflatten(-1, (DV // GROUP, GROUP))      # 64 bits: quotients next to a border between two codes
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
    B, most, total = len(npages), max(1, max(npages)), sum(npages) + spare
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    n = torch.tensor(npages, device=dev)
    k = torch.arange(most, device=dev)
    used = k < n[:, None]
    at = (torch.cumsum(n, 0) - n)[:, None] + k
    return torch.where(used, perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)), total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    span = case["N"] * case["P"]
    if case["kind"] == "decode":
        lens = _lens(case)
        s["bt"], s["pages"] = _table(g, [max(1, -(-x // span)) for x in lens], 0, dev)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int64, device=dev)
        rows = s["pages"] * case["P"]
        s["arena"] = torch.empty(case["held"], rows, ROW, dtype=torch.uint8, device=dev)
        for r in range(case["held"]):
            for a in range(0, rows, 1 << 20):
                x = torch.randn(min(1 << 20, rows - a), DK, generator=g, device=dev).to(torch.bfloat16)
                s["arena"][r, a:a + (1 << 20)] = _pack(x)
        rows = (case["B"], case["q_len"], case["H"])
        s["q"] = torch.randn(*rows, DK, generator=g, device=dev).to(torch.bfloat16)
        s["o"] = torch.empty(case["held"], *rows, DV, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(case["held"], *rows, dtype=torch.float32, device=dev)
    elif case["kind"] in ("append", "relayout"):
        if case["kind"] == "append":
            first = [case["start"] + b for b in range(case["B"])]
            last = [a + case["tokens"] for a in first]
        else:
            first, last = [0] * case["B"], [case["S"] - b for b in range(case["B"])]
        s["bt"], s["pages"] = _table(g, [-(-x // span) for x in last], 3, dev)
        pos = torch.cat([torch.arange(a, e, device=dev) for a, e in zip(first, last)])
        req = torch.cat([torch.full((e - a,), b, dtype=torch.int32, device=dev)
                         for b, (a, e) in enumerate(zip(first, last))])
        if case["kind"] == "append":
            pad = torch.full((case["pad"],), -1, device=dev)
            s["pos"], s["req"] = torch.cat([pos, pad]), torch.cat([req, pad.to(torch.int32)])
            s["rows"] = torch.randn(s["pos"].numel(), DK, generator=g, device=dev).to(torch.bfloat16)
        else:
            s["pos"], s["req"] = pos, req
            s["src_bt"], n = _table(g, [-(-x // case["Ps"]) for x in last], 0, dev)
            s["src"] = torch.randn(n * case["Ps"], DK, generator=g, device=dev).to(torch.bfloat16)
        s["arena"] = torch.zeros(case["held"], s["pages"] * case["P"], ROW, dtype=torch.uint8, device=dev)
        s["kv"] = torch.zeros(s["pos"].numel(), DK, dtype=torch.bfloat16, device=dev)
    else:
        old, new = _lens(case), _grown(case)
        most = max(-(-n // span) for n in new)
        need = sum(-(-n // span) for n in new)
        held = [-(-a // span) for a in old]
        bt, s["pages"] = _table(g, held, need - sum(held) + 5, dev)
        s["bt"] = torch.full((case["B"], most), -1, dtype=torch.int32, device=dev)
        if sum(held):
            s["bt"][:, :bt.shape[1]] = bt
        free = torch.ones(s["pages"] + 1, dtype=torch.bool, device=dev)
        free[s["bt"].flatten().long()] = False          # -1 marks the place behind the last page
        free = torch.nonzero(free[:-1]).flatten().to(torch.int32)
        free = free[torch.randperm(free.numel(), generator=g, device=dev)]
        s["free"] = torch.full((s["pages"],), -1, dtype=torch.int32, device=dev)
        head = s["pages"] // 3
        s["free"][(head + torch.arange(free.numel(), device=dev)) % s["pages"]] = free
        s["free_state"] = torch.tensor([head, free.numel()], dtype=torch.int64, device=dev)
        s["seq_lens"] = torch.tensor(old, dtype=torch.int64, device=dev)
        s["old"], s["new"] = s["seq_lens"].clone(), torch.tensor(new, dtype=torch.int64, device=dev)
        T = sum(new) - sum(old) + 3                     # a buffer a little longer than the step
        for name, dt in (("pos", torch.int64), ("req", torch.int32), ("owner", torch.int32), ("row", torch.int64),
                         ("slot", torch.int64)):
            s[name] = torch.empty(T, dtype=dt, device=dev)
        s["cu"] = torch.empty(case["B"] + 1, dtype=torch.int64, device=dev)
        s["cu_back"] = torch.empty_like(s["cu"])
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- plain forms
def _place(s, pos, req):
    """(owner, local row, slot) of tokens; slot -1 where there is no token."""
    N, I, P = s["N"], s["I"], s["P"]
    owner = torch.where(pos >= 0, (pos // I) % N, -1)
    row = torch.where(pos >= 0, (pos // (N * I)) * I + pos % I, -1)
    page = s["bt"][req.clamp(min=0).long(), (row.clamp(min=0)) // P].long()
    return owner, row, torch.where(pos >= 0, page * P + row % P, -1)


def _decode_plain(s):
    N, I, P, n, B, q_len, H = (s[k] for k in ("N", "I", "P", "held", "B", "q_len", "H"))
    dev = s["q"].device
    L = s["bt"].shape[1] * P
    k = torch.arange(L, device=dev)
    slot = s["bt"].clamp(min=0).long()[:, k // P] * P + k % P                         # [B, L]
    kv = _unpack(s["arena"][:, slot])                                                 # [n, B, L, 576]
    q = s["q"].float().view(B, q_len * H, DK)
    x = torch.matmul(q, kv.transpose(-1, -2)) * SCALE                                 # [n, B, R, L]
    shard = torch.arange(n, device=dev)[:, None]
    at = (k // I * N + shard) * I + k % I                                             # [n, L] positions
    last = s["seq_lens"][:, None] - q_len + torch.arange(q_len, device=dev)           # [B, q_len]
    seen = at[:, None, None, :] <= last[None, :, :, None]                             # [n, B, q_len, L]
    x = x.view(n, B, q_len, H, L).masked_fill_(~seen.unsqueeze(3), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, B, q_len * H, L), kv[..., :DV]).view(n, B, q_len, H, DV)
    lse = (m + torch.log(z)).squeeze(-1)
    s["o"].copy_(o / torch.where(z > 0, z, torch.ones_like(z)))
    s["lse"].copy_(lse * LOG2E if s["base"] else lse)
    return {"o": s["o"], "lse": s["lse"]}


def _store_plain(s, rows):
    owner, _, slot = _place(s, s["pos"], s["req"])
    mine = (owner >= 0) & (owner < s["held"])
    size = s["arena"].shape[1]
    flat = s["arena"].view(-1, ROW)
    at = torch.where(mine, owner * size + slot, 0)
    keep = flat[at]
    first = torch.argmax(mine.to(torch.int32))                                        # entries that are not held
    data = torch.where(mine[:, None], _pack(rows), keep)                              # repeat the first held one
    flat[torch.where(mine, at, at[first])] = torch.where(mine[:, None], data, data[first])
    s["kv"].copy_(torch.where(mine[:, None], _unpack(flat[at]).to(torch.bfloat16), s["kv"]))
    return {"kv": s["kv"]}


def _relayout_plain(s):
    at = s["src_bt"][s["req"].long(), s["pos"] // s["Ps"]].long() * s["Ps"] + s["pos"] % s["Ps"]
    return _store_plain(s, s["src"][at])


def _update_plain(s, new):
    """Block table, free list and lengths of a step to the lengths `new`; the new tokens' prefix sums."""
    old, span, size = s["seq_lens"], s["N"] * s["P"], s["free"].numel()
    before, after = (old + span - 1) // span, (new + span - 1) // span
    k = torch.arange(s["bt"].shape[1], device=new.device)
    take = (k >= before[:, None]) & (k < after[:, None])
    give = (k >= after[:, None]) & (k < before[:, None])
    nth = torch.cumsum(take.flatten().long(), 0).view_as(take) - 1
    back = torch.cumsum(give.flatten().long(), 0).view_as(give) - 1
    head, count = s["free_state"][0], s["free_state"][1]
    ring = torch.cat([s["free"], s["free"][:1]])                                      # one place for what is not given back
    ring[torch.where(give, (head + count + back) % size, size)] = s["bt"]
    table = torch.where(take, s["free"][(head + nth.clamp(min=0)) % size], s["bt"])
    s["bt"].copy_(torch.where(give, -1, table))
    s["free"].copy_(ring[:-1])
    s["free_state"].copy_(torch.stack([(head + take.sum()) % size, count - take.sum() + give.sum()]))
    more = torch.cumsum((new - old).clamp(min=0), 0)
    s["seq_lens"].copy_(new)
    return torch.cat([torch.zeros_like(more[:1]), more])


def _tables_plain(s):
    old = s["seq_lens"].clone()
    s["cu"].copy_(_update_plain(s, s["new"]))
    t = torch.arange(s["pos"].numel(), device=old.device)
    req = torch.searchsorted(s["cu"][1:], t, right=True)
    here = req < s["B"]
    req = req.clamp(max=s["B"] - 1)
    s["pos"].copy_(torch.where(here, old[req] + t - s["cu"][req], -1))
    s["req"].copy_(torch.where(here, req, -1))
    owner, row, slot = _place(s, s["pos"], s["req"])
    s["owner"].copy_(owner)
    s["row"].copy_(row)
    s["slot"].copy_(slot)
    s["cu_back"].copy_(_update_plain(s, s["old"]))
    return _tables_out(s)


def _tables_out(s):
    return {k: s[k] for k in ("pos", "req", "owner", "row", "slot", "cu", "cu_back", "bt", "free", "free_state", "seq_lens")}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    import context_sharded_mla_gb300 as dcp

    lay = dcp.Layout(s["N"], s["I"], s["P"])
    if s["kind"] == "decode":
        if "ws" not in s:                               # kept by a program beside its buffers
            size = dcp.dcp_mla_decode_workspace_size_q4(lay, 0, s["held"], s["B"], s["q_len"], s["H"])
            s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=s["q"].device)
        dcp.dcp_mla_decode_partial_q4(lay, 0, s["held"], s["q"], s["arena"], s["pages"], s["bt"], s["bt"].shape[1],
                                      s["seq_lens"], SCALE, dcp.DCP_LSE_BASE_2 if s["base"] else dcp.DCP_LSE_BASE_E,
                                      s["o"], s["lse"], s["ws"], s["status"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["kind"] in ("append", "relayout"):
        if s["kind"] == "append":
            dcp.dcp_kv_append_q4(lay, 0, s["held"], s["rows"], s["pos"], s["req"], s["bt"], s["bt"].shape[1],
                                 s["arena"], s["pages"], s["status"])
        else:
            dcp.dcp_kv_relayout_q4(lay, 0, s["held"], s["src"], s["Ps"], s["src_bt"], s["src_bt"].shape[1], s["pos"],
                                   s["req"], s["bt"], s["bt"].shape[1], s["arena"], s["pages"], s["status"])
        dcp.dcp_kv_read_q4(lay, 0, s["held"], s["arena"], s["pages"], s["pos"], s["req"], s["bt"], s["bt"].shape[1],
                           s["kv"], s["status"])
        return {"kv": s["kv"]}
    dcp.dcp_block_tables(lay, s["seq_lens"], s["new"], s["bt"], s["bt"].shape[1], s["free"], s["free_state"], s["cu"],
                         s["status"], pos=s["pos"], req=s["req"], owner=s["owner"], row=s["row"], slot=s["slot"])
    dcp.dcp_block_tables(lay, s["seq_lens"], s["old"], s["bt"], s["bt"].shape[1], s["free"], s["free_state"],
                         s["cu_back"], s["status"])
    return _tables_out(s)


def run(state):
    if own:
        return _own(state)
    if state["kind"] == "decode":
        return _decode_plain(state)
    if state["kind"] == "append":
        return _store_plain(state, state["rows"])
    if state["kind"] == "relayout":
        return _relayout_plain(state)
    return _tables_plain(state)


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
    """What the cache holds of bf16 rows, in 64 bits: the scale by search among all e4m3 values, codes by comparison."""
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


def exact(case, seed):
    if case["kind"] == "tables":
        return None
    s = prepare(case, seed)
    N, I, P = case["N"], case["I"], case["P"]
    if case["kind"] == "decode":
        n, B, q_len, H = case["held"], case["B"], case["q_len"], case["H"]
        o = torch.zeros(n, B, q_len, H, DV, dtype=torch.float64, device=s["q"].device)
        lse = torch.full((n, B, q_len, H), -math.inf, dtype=torch.float64, device=s["q"].device)
        for b, S in enumerate(_lens(case)):
            p = torch.arange(S, device=s["q"].device)
            for r in range(n):
                at = p[(p // I) % N == r]
                if not at.numel():
                    continue
                local = at // (N * I) * I + at % I
                kv = _exact_rows(s["arena"][r, s["bt"][b, local // P].long() * P + local % P])
                x = s["q"][b].double().flatten(0, 1) @ kv.T / math.sqrt(192.0)
                x = x.view(q_len, H, -1)
                x = x.masked_fill(at[None, None, :] > S - q_len + torch.arange(q_len, device=at.device)[:, None, None],
                                  -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z).unsqueeze(-1))
                o[r, b] = (w.flatten(0, 1) @ kv[:, :DV]).view(q_len, H, DV)
                lse[r, b] = z / math.log(2.0) if case["base"] else z
        return {"o": o, "lse": lse}
    if case["kind"] == "append":
        rows = s["rows"]
    else:
        b = s["req"].long()
        rows = s["src"][s["src_bt"][b, s["pos"] // case["Ps"]].long() * case["Ps"] + s["pos"] % case["Ps"]]
    mine = (s["pos"] >= 0) & (s["pos"] // I % N < case["held"])
    return {"kv": torch.where(mine[:, None], _exact_values(rows), torch.zeros_like(rows).double())}
