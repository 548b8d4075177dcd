"""Oracle: attention weight of cached rows, the rows that stay and their move (fp64, CPU).

TEST INFRASTRUCTURE ONLY (see the package docstring).

The weight of a key is its softmax probability under the merged lse, summed over the
query rows that see it.  A shard keeps count(new length) of its own rows ("PCP / DCP：
计算、KV 布局与块轮转", section 6, local_len): sinks, then recent rows, then by weight.
"""

from __future__ import annotations

import numpy as np

from . import layout


def key_weights(q, kv, S, scale, lse, base):
    """(weights [S], their error scale [S]) of one request: q [q_len, H, 576], kv [S, 576] in position order, lse
    [q_len, H] in base e (0) or base 2 (1).  The second sums each term times 1 + |score| + |lse|."""
    q_len, H, _ = q.shape
    s = (q.reshape(-1, q.shape[-1]) @ kv.T).reshape(q_len, H, S) * scale
    z = np.asarray(lse, np.float64) * (np.log(2.0) if base else 1.0)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(np.isneginf(z)[..., None], 0.0, np.exp(s - z[..., None]))
    seen = np.arange(S)[None, :] <= (S - q_len + np.arange(q_len))[:, None]
    e = np.where(seen[:, None, :], e, 0.0)
    size = np.where(seen[:, None, :], 1 + np.abs(s) + np.where(np.isfinite(z), np.abs(z), 0)[..., None], 0.0)
    return e.sum((0, 1)), (e * size).sum((0, 1))


def select(weights, r, S, new, N, I, sinks, recent):
    """Rows shard r keeps (ascending), one row at a time from the sequence's definition."""
    n, m = int(layout.count(r, S, N, I)), int(layout.count(r, new, N, I))
    pos = [int(layout.global_pos(r, i, N, I)) for i in range(n)]
    first = [i for i in range(n) if pos[i] < sinks]
    late = [i for i in range(n - 1, -1, -1) if pos[i] >= sinks and pos[i] >= S - recent]
    taken = set(first) | set(late)
    rest = [i for i in range(n) if i not in taken]
    rest.sort(key=lambda i: (0 if np.isnan(weights[i]) else 1, -weights[i] if not np.isnan(weights[i]) else 0.0, i))
    return sorted((first + late + rest)[:m])
