"""Root-mean-square norm of rows with the residual's addition in front:
h = x + r, y = h * w / sqrt(mean(h^2) + eps); 8-bit output s = max|y| / 127,
q = round(y / s) (0 for an all-zero row).

Test infrastructure only (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def rmsnorm_f64(x: np.ndarray, weight: np.ndarray, eps: float, residual=None):
    """(h, y) in f64 for rows along the last axis."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    mean = np.sum(h * h, axis=-1, keepdims=True) / x.shape[-1]
    return h, h * weight.astype(np.float64) / np.sqrt(mean + eps)


def quantise_f64(y: np.ndarray):
    """(q, s) of the 8-bit output in f64."""
    s = np.abs(y).max(axis=-1) / 127.0
    return np.where(s[..., None] > 0, np.rint(y / np.where(s > 0, s, 1.0)[..., None]), 0.0), s
