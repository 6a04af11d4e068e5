"""Block-scaled e4m3 in fp64: the quantization and the values that codes and
scales stand for, from the format's definition (the pages name blockwise FP8
linear layers, report page, part 6/7, section 4.3 "Cost Estimation", and the
model card "Puro", section "Training", without a rounding or a scale type).

  grid: 0, m * 2^-9 (m = 1..7), (8 + m) * 2^(e - 10) (e = 1..15, m = 0..7)
        without (15, 7), which is NaN: largest 448.
  scale of a block with largest finite magnitude a: 2^e, e the smallest
        integer >= -126 with a <= 448 * 2^e.
  code: the grid value nearest to x / 2^e, ties to the even code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def grid() -> np.ndarray:
    """Values of the codes 0 .. 126."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(1.0 * m, -9))


def decode(codes: np.ndarray) -> np.ndarray:
    v = np.append(grid(), np.nan)[codes & 127]
    return np.where(codes & 128, -v, v)


def encode(v: np.ndarray) -> np.ndarray:
    """fp64 values of magnitude at most 448 (or not finite: NaN codes) to the
    nearest code; which NaN code is left open, here 127 with the sign."""
    g = grid()
    a = np.abs(v)
    hi = np.clip(np.searchsorted(g, np.where(np.isfinite(a), a, 0.0)), 1, 126)
    lo = hi - 1
    dl, dh = np.where(np.isfinite(a), a, 0.0) - g[lo], g[hi] - np.where(np.isfinite(a), a, 0.0)
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isfinite(a), c, 127)
    return (c | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _pad(v: int, m: int) -> int:
    return -(-v // m) * m


def quantize(x: np.ndarray, block: str = "rows"):
    """(codes, scale bytes) in the stored layout: codes rows x (cols up to a
    multiple of 128), zeros past cols; scales (rows or tile rows) x (blocks up
    to a multiple of 4), zeros past the last block."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    br = BLOCK if block == "tiles" else 1
    nr, nc = -(-rows // br), -(-cols // BLOCK)
    p = np.zeros((nr * br, nc * BLOCK))
    p[:rows, :cols] = x
    b = p.reshape(nr, br, nc, BLOCK)
    a = np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=(1, 3), initial=0.0)
    e = np.full(a.shape, -126)
    while np.any(bad := a > np.ldexp(448.0, e)):   # one step of two at a time, from below
        e = np.where(bad, e + 1, e)
    with np.errstate(invalid="ignore"):
        codes = encode(b / np.ldexp(1.0, e)[:, None, :, None]).reshape(nr * br, nc * BLOCK)[:rows]
    scales = np.zeros((nr, _pad(nc, 4)), np.uint8)
    scales[:, :nc] = e + 127
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, shape, block: str = "rows") -> np.ndarray:
    rows, cols = shape
    br = BLOCK if block == "tiles" else 1
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    i, j = np.arange(rows) // br, np.arange(cols) // BLOCK
    return decode(codes[:, :cols]) * s[np.ix_(i, j)]
