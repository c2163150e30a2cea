"""Attention of one new token per sequence over a paged cache:
o = sum_l p_l v_l / sum_l p_l with p_l = exp(scale q.k_l), grouped heads;
zeros for a sequence without tokens.

Test infrastructure only (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def gather(pool: np.ndarray, pages: np.ndarray, n: int) -> np.ndarray:
    """The first n rows of a sequence, [n][kv_heads][dim], from pool [pages][page][kv_heads][dim]."""
    page = pool.shape[1]
    return np.stack([pool[pages[t // page], t % page] for t in range(n)]) if n else np.zeros((0,) + pool.shape[2:])


def attend_f64(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """(o, sum_l w_l |v_l|, largest sum_d |q_d k_ld| * scale) for q [heads][dim] over k, v [n][kv_heads][dim]."""
    H, D = q.shape
    o, S, Q = np.zeros((H, D)), np.zeros((H, D)), np.zeros(H)
    if k.shape[0] == 0:
        return o, S, Q
    group = H // k.shape[1]
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    for h in range(H):
        kh, vh = k[:, h // group], v[:, h // group]
        s = scale * (kh @ q[h])
        p = np.exp(s - s.max())
        p /= p.sum()
        o[h], S[h] = p @ vh, p @ np.abs(vh)
        Q[h] = abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
    return o, S, Q
