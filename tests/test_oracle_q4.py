"""Pins of the 4-bit cache oracle and the block-table oracle (no GPU)."""

import itertools
import random

import numpy as np
import pytest

from oracle import cache_q4, layout, tables


def test_e4m3_table():
    assert cache_q4.E4M3[0] == 0 and cache_q4.E4M3[1] == 2.0 ** -9 and cache_q4.E4M3[126] == 448
    assert cache_q4.E4M3[8] == 2.0 ** -6 and cache_q4.E4M3[0x38] == 1.0
    assert np.all(np.diff(cache_q4.E4M3) > 0)


def test_quantise_closed_forms():
    x = np.arange(-8, 8) * 0.25                      # largest magnitude 2: 2/7 lies next to 0.28125
    codes, s = cache_q4.quantise_group(x)
    assert cache_q4.E4M3[s] == 0.28125
    assert codes.tolist() == [-7, -6, -5, -4, -4, -3, -2, -1, 0, 1, 2, 3, 4, 4, 5, 6]
    x = np.full(16, 0.5)
    x[0] = 7.0                                       # scale 1: 0.5 is a tie and goes to the even code 0
    codes, s = cache_q4.quantise_group(x)
    assert cache_q4.E4M3[s] == 1.0 and codes.tolist() == [7] + [0] * 15
    x[1:] = 1.5                                      # ... and 1.5 to 2
    assert cache_q4.quantise_group(x)[0].tolist() == [7] + [2] * 15
    assert cache_q4.quantise_group(np.zeros(16))[1] == 0
    assert cache_q4.quantise_group(np.full(16, 1e6))[1] == 126
    tiny = np.full(16, 7 * 2.0 ** -10)               # half of the smallest scale: a tie, to 0
    assert cache_q4.quantise_group(tiny)[1] == 0
    assert cache_q4.quantise_group(tiny * (1 + 2.0 ** -7))[1] == 1


def test_error_is_at_most_half_a_step_of_the_scale():
    rng = np.random.default_rng(0)
    for x in rng.standard_normal((200, 16)):
        codes, s = cache_q4.quantise_group(x)
        step = cache_q4.E4M3[s]
        # the scale is within 1/16 of max/7, so 7 steps reach at least 15/16 of the maximum
        assert np.all(np.abs(codes * step - x) <= np.maximum(step / 2, np.abs(x) / 16) + 1e-15)


def test_pack_unpack_round_trip():
    rng = np.random.default_rng(1)
    codes = rng.integers(-8, 8, (5, 512))
    scales = rng.integers(0, 127, (5, 32)).astype(np.uint8)
    rope = rng.integers(0, 0x7F00, (5, 64)).astype(np.uint16)
    rows = cache_q4.pack(codes, scales, rope)
    assert rows.shape == (5, cache_q4.ROW_BYTES)
    got = cache_q4.unpack(rows)
    assert np.array_equal(got[:, :512], codes * np.repeat(cache_q4.E4M3[scales], 16, axis=1))
    assert np.array_equal(got[:, 512:], (rope.astype(np.uint32) << 16).view(np.float32).astype(np.float64))
    # dim 8k + 2i sits in bits 4i, its neighbour 16 bits above
    one = np.full((1, 512), -8)
    one[0, 5] = -7
    assert cache_q4.pack(one, scales[:1], rope[:1])[0, :4].view("<u4")[0] == 1 << 24


def test_values_fit_bf16():
    """A code times an e4m3 scale has at most 7 significant bits, so bf16 holds it."""
    v = (np.arange(-8, 8)[:, None] * cache_q4.E4M3[None]).astype(np.float32)
    assert np.all((v.view(np.uint32) & 0xFFFF) == 0)


@pytest.mark.parametrize("N,I,P", [(1, 1, 8), (4, 1, 16), (3, 2, 8), (2, 8, 8)])
def test_tables_hold_every_position_once(N, I, P):
    """Through random steps: every held position has a slot of its own, no page is lost or held twice."""
    rng = random.Random(N * 100 + I * 10 + P)
    B, cap, most = 5, 40, 9
    lens, table = [0] * B, [[-1] * most for _ in range(B)]
    ring, head, count = list(range(cap)), rng.randrange(cap), cap
    ring = ring[-head:] + ring[:-head] if head else ring
    for _ in range(60):
        new = [rng.choice([0, n, min(n + rng.randrange(1, 3 * N * P), most * N * P), rng.randrange(most * N * P)])
               for n in lens]
        old = list(lens)
        head, count, tokens, cu, status = tables.update(lens, new, table, most, ring, head, count, N, I, P)
        if status:
            assert status == tables.NO_PAGES and lens == old and not tokens
            continue
        assert lens == new
        assert [t[:2] for t in tokens] == [(p, b) for b in range(B) for p in range(old[b], new[b])]
        assert cu == list(itertools.accumulate([0] + [max(0, n - a) for a, n in zip(old, new)]))
        held = [p for row in table for p in row if p >= 0]
        free = [ring[(head + i) % cap] for i in range(count)]
        assert sorted(held + free) == list(range(cap))
        for b in range(B):
            used = -(-new[b] // (N * P))
            assert all(x >= 0 for x in table[b][:used]) and all(x == -1 for x in table[b][used:])
            # one page per shard and N P positions is what the longest shard needs
            assert used == max(-(-int(layout.count(r, new[b], N, I)) // P) for r in range(N))
        if tokens:
            o, r, s = layout.slot_map([t[0] for t in tokens], [t[1] for t in tokens], table, N, I, P)
            assert [t[2:] for t in tokens] == list(zip(map(int, o), map(int, r), map(int, s)))


def test_tables_refuse_as_a_whole():
    def step(lens, new, head=0, count=3, T=None, most=4):
        table, ring = [[9, -1, -1, -1], [-1] * 4], [5, 6, 7, 9]
        got = tables.update(lens, new, table, most, ring, head, count, 2, 1, 8, T)
        return got, table, ring
    got, table, ring = step([3, 0], [17, 40])        # needs 1 + 3 of 3 pages
    assert got[4] == tables.NO_PAGES and table[0] == [9, -1, -1, -1] and ring == [5, 6, 7, 9]
    assert step([3, 0], [3, -1])[0][4] == tables.BAD_LENGTH
    assert step([3, 0], [3, 65])[0][4] == tables.BAD_PAGE_INDEX
    assert step([3, 0], [9, 9], T=14)[0][4] == tables.TOO_MANY_TOKENS
    assert step([3, 0], [0, 0], count=4)[0][4] == tables.BAD_POOL
    got, table, ring = step([3, 0], [0, 17])         # one page back, two taken
    assert got == (2, 2, [(p, 1, p % 2, p // 2, (5 if p < 16 else 6) * 8 + p // 2 % 8) for p in range(17)],
                   [0, 0, 17], 0)
    assert ring == [5, 6, 7, 9] and table == [[-1] * 4, [5, 6, -1, -1]]
