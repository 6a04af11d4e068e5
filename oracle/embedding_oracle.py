"""fp64 oracle of the embedding lookup and its gradient, token by token:

  out[t] = scale * table[ids[t] - first], zeros where that is no row
  G[v] = old G[v] + scale * sum of dy[t] over the t with ids[t] - first = v

Test infrastructure only: shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def lookup(ids: np.ndarray, table: np.ndarray, scale: float, first: int = 0) -> np.ndarray:
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if first <= int(i) < first + len(table):
            out[t] = scale * np.asarray(table[int(i) - first], np.float64)
    return out


def gradient(ids: np.ndarray, dy: np.ndarray, rows: int, scale: float, old=None, first: int = 0):
    """(G, sums of magnitudes and numbers of terms that each row's tolerance counts)."""
    g, size, count = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1])), np.zeros(rows, np.int64)
    for t, i in enumerate(ids):
        if first <= int(i) < first + rows:
            v = scale * np.asarray(dy[t], np.float64)
            g[int(i) - first] += v
            size[int(i) - first] += np.abs(v)
            count[int(i) - first] += 1
    if old is not None:
        g += old
        size += np.abs(old)
    return g, size, count
