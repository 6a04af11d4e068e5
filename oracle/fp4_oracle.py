"""fp64 oracle of microscaled 4-bit matrices (formats of include/muonh.h): e2m1
codes, two to a byte, with a power-of-two scale per 32 entries of a row. Numpy only, from
the definitions: the scale is the smallest 2^e, e >= -126, with max|x| <= 6 * 2^e;
a code is the nearest value to x / 2^e, ties to the even code.

Test infrastructure only: shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(v: np.ndarray) -> np.ndarray:
    """Codes of values of at most 6 in magnitude."""
    a = np.abs(v)
    hi = np.searchsorted(GRID, a)  # the first grid value >= a
    hi = np.minimum(hi, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    pick = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (pick | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    return np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]


def _exponent(a: float) -> int:
    if a == 0:
        return -126
    m, e = np.frexp(a)  # a = m 2^e, 0.5 <= m < 1; 6 = 0.75 * 2^3
    return max(int(e) - 3 + (1 if m > 0.75 else 0), -126)


def quantize(x: np.ndarray):
    """(codes, one to a byte, rows x padded columns; scale bytes, padded)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    ld, sld = -(-cols // 256) * 256, -(-cols // 256) * 8
    codes, scales = np.zeros((rows, ld), np.uint8), np.zeros((rows, sld), np.uint8)
    for r in range(rows):
        for g in range(-(-cols // GROUP)):
            v = x[r, g * GROUP:(g + 1) * GROUP]
            if not np.isfinite(v).all():
                scales[r, g] = 255
                continue
            e = _exponent(np.abs(v).max())
            scales[r, g] = e + 127
            codes[r, g * GROUP:g * GROUP + len(v)] = encode(np.ldexp(v, -e))
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[:, 0::2] | codes[:, 1::2] << 4


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def values(packed: np.ndarray, scales: np.ndarray, shape) -> np.ndarray:
    rows, cols = shape
    e = scales.astype(np.int64).repeat(GROUP, 1)[:, :cols]
    v = np.ldexp(decode(unpack(packed)[:, :cols]), e - 127)
    return np.where(e == 255, np.nan, v)
