"""Oracle: RMS norm and rotation of the position dims (fp64, CPU).

TEST INFRASTRUCTURE ONLY (see the package docstring).

"MLA 的 Decode Context Parallelism", section 2: a cached row is the normalised latent
c_K and the rotated k_R.  A pair of position dims (a, b) is the complex number a + ib;
position p turns it by p * inv_freq[i], i.e. multiplies it by exp(i p inv_freq[i]).
"""

from __future__ import annotations

import numpy as np


def rms_norm(x, gamma, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def rotate(x, pos, inv_freq, halves):
    """x [T, ..., 64] at positions pos [T]: pairs (i, i + 32) if `halves`, else (2i, 2i + 1)."""
    x = np.asarray(x, np.float64)
    i = np.arange(32)
    re, im = (i, i + 32) if halves else (2 * i, 2 * i + 1)
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    z = (x[..., re] + 1j * x[..., im]) * np.exp(1j * angle).reshape(len(x), *([1] * (x.ndim - 2)), 32)
    out = np.empty_like(x)
    out[..., re], out[..., im] = z.real, z.imag
    return out
