"""Oracle for the 4-bit key / value cache -- TEST INFRASTRUCTURE ONLY.

Only the test suite and ``__graft_entry__.smoke()`` may import this module; the
product path never does, and this module imports nothing from the product.

What the format keeps of a row, in float64, straight from its definition: 16
neighbouring elements share s = max|x| / 6 rounded to the nearest scale (5
exponent bits, 3 mantissa bits, no sign, at most 10240; ties to the even one by
index), and each element becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to
|x| / s (ties to the even one by index), with its sign, times s.  A NaN counts
as 0.  The division is exact enough in float64: |x| and s have at most 24 and 4
significant bits, so |x| / s is a border between two values or differs from it
by more than 2^-26 of itself.
"""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
SCALES = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 18)
                   for e in range(31) for m in range(8)])
SCALES = SCALES[SCALES <= 10240]


def nearest(x, values):
    """Index of the nearest of the sorted ``values``; of two as near the even index."""
    mid = (values[1:] + values[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, "left"), np.searchsorted(mid, x, "right")
    return np.where(lo % 2 == 0, lo, hi)


def kept(x):
    """What the cache holds of rows ``x`` (..., d), d a multiple of 16, float64."""
    x = np.asarray(x, dtype=np.float64)
    g = np.where(np.isnan(x), 0.0, x).reshape(-1, 16)
    s = SCALES[nearest(np.minimum(np.abs(g).max(axis=1), 61440) / 6, SCALES)][:, None]
    with np.errstate(invalid="ignore", divide="ignore"):
        r = np.where(s > 0, np.abs(g) / s, 0.0)
    return (np.sign(g) * LEVELS[nearest(r, LEVELS)] * s).reshape(x.shape)


def unpack_tile(tile, dk, dv):
    """Keys (16, dk) and values (16, dv) of one tile's bytes, element by element."""
    tile = np.asarray(tile, dtype=np.int64)

    def value(byte, nibble, scale):
        c = (tile[byte] >> (4 * nibble)) & 15
        return LEVELS[c & 7] * (-1.0 if c & 8 else 1.0) * SCALES[tile[scale]]

    k, v = np.zeros((16, dk)), np.zeros((16, dv))
    part = min(dk, 128)
    for t in range(16):
        for x in range(dk):
            c, y = divmod(x, part)
            k[t, x] = value(c * 8 * part + t * part // 2 + y // 2, y % 2,
                            8 * dk + c * part + t * part // 16 + y // 16)
    n = min(16, dv // 8)
    for t in range(16):
        for x in range(dv):
            c, y = divmod(x, 128)
            g, z = divmod(y, n)
            r = 2 * c + z // 8
            byte = (((r * 8 + g) * 4 + t // 4) * 4 + z % 8 // 2) * 4 + 2 * (t % 4 // 2) + z % 2
            v[t, x] = value(9 * dk + byte, t % 2, 9 * dk + 8 * dv + x // 16 * 16 + t)
    return k, v
