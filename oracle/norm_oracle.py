"""fp64 oracle of RMS norm with the residual's addition, forward and backward,
written from the formulas:

  h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  y = h r w
  n = h r, g = dy w:  dh = r (g - n mean(g n)) + dresidual;  dw = sum over rows of dy n

Test infrastructure only: shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def forward(h: np.ndarray, w: np.ndarray, eps: float):
    """(y, r) of the rows of h (which holds x + residual)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * r[:, None] * w, r


def backward(dy: np.ndarray, h: np.ndarray, w: np.ndarray, r: np.ndarray, dresidual=None):
    """(dh, dw)."""
    dy, h, w, r = (np.asarray(v, np.float64) for v in (dy, h, w, r))
    n, g = h * r[:, None], dy * w
    dh = r[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return dh if dresidual is None else dh + np.asarray(dresidual, np.float64), np.sum(dy * n, axis=0)
