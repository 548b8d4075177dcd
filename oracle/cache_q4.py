"""Oracle: the 4-bit latent cache (quantisation, byte layout), in fp64 and integers.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A group of 16 dims x with largest magnitude A is held as scale = the e4m3 value
nearest to min(A / 7, 448) and codes = the integers nearest to x / scale, clamped
to [-7, 7] (0 where the scale is 0), ties to even in both.  A row of 576 dims is
416 bytes: 64 words of codes (word k: dim 8k + 2i in bits [4i, 4i + 4), dim
8k + 2i + 1 in bits [16 + 4i, 20 + 4i), each plus 8), 32 e4m3 scales, 64 bf16.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

GROUP, ROW_BYTES = 16, 416

# e4m3 bit patterns 0 .. 126 (127 is NaN) in increasing order of value
E4M3 = np.array([(1 + (e & 7) / 8) * 2.0 ** ((e >> 3) - 7) if e >= 8 else e / 512 for e in range(127)])


def _nearest_scale(v: Fraction) -> int:
    """Bit pattern of the e4m3 value nearest to v >= 0 (ties to the even pattern, at most 448)."""
    if v >= Fraction(448):
        return 126
    hi = int(np.searchsorted(E4M3, float(v)))
    hi = min(max(hi, 1), 126)
    while Fraction(E4M3[hi]) < v:
        hi += 1
    while hi > 1 and Fraction(E4M3[hi - 1]) >= v:
        hi -= 1
    a, b = v - Fraction(E4M3[hi - 1]), Fraction(E4M3[hi]) - v
    if a != b:
        return hi - 1 if a < b else hi
    return hi - 1 if (hi - 1) % 2 == 0 else hi


def quantise_group(x):
    """(codes int[16], scale bit pattern) of 16 finite values, in rational arithmetic."""
    q = [Fraction(float(v)) for v in x]
    s = _nearest_scale(max(abs(v) for v in q) / 7)
    if s == 0:
        return np.zeros(GROUP, np.int64), 0
    step = Fraction(E4M3[s])
    # round() of a Fraction goes to the nearest integer, ties to even
    return np.array([min(7, max(-7, round(v / step))) for v in q], np.int64), s


def quantise(x):
    """(codes int[..., 512], scale patterns uint8[..., 32]) of values [..., 512]."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.shape, np.int64)
    scales = np.zeros(x.shape[:-1] + (32,), np.uint8)
    for at in np.ndindex(*scales.shape):
        sl = at[:-1] + (slice(GROUP * at[-1], GROUP * (at[-1] + 1)),)
        codes[sl], scales[at] = quantise_group(x[sl])
    return codes, scales


def pack(codes, scales, rope_bits):
    """Row bytes uint8[..., 416] from codes [..., 512], scale patterns [..., 32], bf16 patterns [..., 64]."""
    lead = codes.shape[:-1]
    words = np.zeros(lead + (64,), np.uint32)
    for d in range(512):
        k, j = divmod(d, 8)
        words[..., k] |= ((codes[..., d] + 8).astype(np.uint32)) << np.uint32(4 * (j // 2) + 16 * (j % 2))
    return np.concatenate([np.ascontiguousarray(words.astype("<u4")).view(np.uint8).reshape(lead + (256,)), scales,
                           np.ascontiguousarray(rope_bits.astype("<u2")).view(np.uint8).reshape(lead + (128,))], -1)


def unpack(rows):
    """The fp64 values [..., 576] of row bytes uint8[..., 416]."""
    rows = np.ascontiguousarray(rows, dtype=np.uint8)
    lead = rows.shape[:-1]
    words = np.ascontiguousarray(rows[..., :256]).view("<u4").reshape(lead + (64,)).astype(np.int64)
    out = np.zeros(lead + (576,))
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    scale = table[rows[..., 256:288]]
    for d in range(512):
        k, j = divmod(d, 8)
        code = ((words[..., k] >> (4 * (j // 2) + 16 * (j % 2))) & 15) - 8
        out[..., d] = code * scale[..., d // GROUP]
    rope = np.ascontiguousarray(rows[..., 288:]).view("<u2").reshape(lead + (64,)).astype(np.uint32) << np.uint32(16)
    out[..., 512:] = rope.astype("<u4").view("<f4")
    return out
