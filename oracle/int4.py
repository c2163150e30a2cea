"""4-bit weights with group scales: w[r][c] = s[r][g] * (q[r][c] - z[r][g]),
g = c // group, the low four bits of code byte j holding column 2j; z = 8
where no zero points are given.

Test infrastructure only (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def decode_f64(code: np.ndarray, scale: np.ndarray, zero, group: int) -> np.ndarray:
    R, C = code.shape[0], 2 * code.shape[1]
    q = np.empty((R, C), dtype=np.float64)
    for c in range(C):
        q[:, c] = (code[:, c // 2] >> (4 * (c % 2))) & 15
    w = np.empty((R, C), dtype=np.float64)
    for g in range(C // group):
        cols = slice(g * group, (g + 1) * group)
        z = 8.0 if zero is None else zero[:, g: g + 1].astype(np.float64)
        w[:, cols] = scale[:, g: g + 1].astype(np.float64) * (q[:, cols] - z)
    return w
