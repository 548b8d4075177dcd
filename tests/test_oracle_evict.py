"""Pins of the eviction and norm/rotation oracle: brute force, invariants, hand-made cases (no GPU)."""

import math

import numpy as np
import pytest

from oracle import attention, evict, layout, norm_rope


def test_key_weights_sum_to_the_query_rows_and_match_a_loop():
    rng = np.random.default_rng(1)
    S, q_len, H = 23, 3, 2
    q, kv = rng.standard_normal((q_len, H, 576)), rng.standard_normal((S, 576))
    lse = np.full((q_len, H), -np.inf)
    want = np.zeros(S)
    for t in range(q_len):
        for h in range(H):
            s = [sum(q[t, h] * kv[p]) * 0.07 for p in range(S - q_len + t + 1)]
            lse[t, h] = math.log(sum(math.exp(x) for x in s))
            for p, x in enumerate(s):
                want[p] += math.exp(x - lse[t, h])
    got, _ = evict.key_weights(q, kv, S, 0.07, lse, 0)
    assert np.allclose(got, want, rtol=1e-12) and abs(got.sum() - q_len * H) < 1e-12
    got2, _ = evict.key_weights(q, kv, S, 0.07, lse / math.log(2), 1)
    assert np.allclose(got2, got, rtol=1e-12)
    o, z, _, _ = attention.sharded_attention(q, kv, S, 4, 1, 0.07, 0)   # the merged lse is that of unsharded attention
    assert np.allclose(np.asarray(z).reshape(q_len, H), lse, atol=1e-12)


@pytest.mark.parametrize("N,I", [(1, 1), (4, 1), (3, 2)])
def test_select_keeps_the_layouts_share(N, I):
    rng = np.random.default_rng(2)
    S = 61
    for new in (0, 1, 7, 30, 60, 61):
        total = 0
        for r in range(N):
            w = rng.random(S)
            kept = evict.select(w, r, S, new, N, I, 4, 9)
            assert len(kept) == layout.count(r, new, N, I) and kept == sorted(set(kept))
            total += len(kept)
        assert total == new


def test_select_order_by_hand():
    w = np.array([0.0, 5.0, 1.0, 1.0, np.nan, 1.0, 0.5, 9.0])
    pick = lambda new, sinks, recent: evict.select(w, 0, 8, new, 1, 1, sinks, recent)   # noqa: E731
    assert pick(2, 0, 0) == [4, 7] and pick(3, 0, 0) == [1, 4, 7]
    assert pick(4, 0, 0) == [1, 2, 4, 7] and pick(5, 0, 0) == [1, 2, 3, 4, 7]      # ties: the lowest row
    assert pick(3, 1, 2) == [0, 6, 7] and pick(2, 1, 2) == [0, 7] and pick(1, 1, 2) == [0]
    assert pick(4, 1, 2) == [0, 4, 6, 7] and pick(8, 20, 20) == list(range(8)) and pick(3, 20, 20) == [0, 1, 2]


def test_rotation_and_norm():
    x = np.zeros((2, 64))
    x[:, 0], x[:, 3] = 1.0, 2.0
    f = np.linspace(0.3, 0.9, 32)
    y = norm_rope.rotate(x, [0, 5], f, False)
    assert np.allclose(y[0], x[0])
    assert np.allclose(y[1, :4], [math.cos(5 * f[0]), math.sin(5 * f[0]), -2 * math.sin(5 * f[1]), 2 * math.cos(5 * f[1])])
    y = norm_rope.rotate(x, [0, 5], f, True)
    assert np.allclose([y[1, 0], y[1, 32], y[1, 3], y[1, 35]],
                       [math.cos(5 * f[0]), math.sin(5 * f[0]), 2 * math.cos(5 * f[3]), 2 * math.sin(5 * f[3])])
    # scores depend on the distance alone
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    for halves in (False, True):
        s = [float((norm_rope.rotate(a, [p], f, halves) * norm_rope.rotate(b, [p + 7], f, halves)).sum()) for p in (0, 1000003)]
        assert abs(s[0] - s[1]) < 1e-8
    n = norm_rope.rms_norm(np.array([[3.0, -4.0]]), [1.0, 2.0], 0.0)
    assert np.allclose(n, [[3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]])
