"""Rows of a paged key-value cache: the position rotation, groups in 4 bits and
the bounds of blocks.

Test infrastructure only (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def angles_f32(rot: int, positions: int, base: float = 10000.0) -> np.ndarray:
    """cos and sin, fp32 [positions][rot / 2][2]."""
    out = np.empty((positions, rot // 2, 2), dtype=np.float32)
    for i in range(rot // 2):
        a = np.arange(positions, dtype=np.float64) * base ** (-2.0 * i / rot)
        out[:, i, 0], out[:, i, 1] = np.cos(a), np.sin(a)
    return out


def turn_f64(x: np.ndarray, angles: np.ndarray, interleaved: bool):
    """(y, |terms|) for rows x [n][heads][dim] with their positions' angles [n][rot / 2][2]."""
    y, mag = x.astype(np.float64), np.abs(x.astype(np.float64))
    half = angles.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = (angles[:, i, j].astype(np.float64)[:, None] for j in (0, 1))
        u, w = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
        y[..., a], y[..., b] = u * c - w * s, w * c + u * s
        mag[..., a], mag[..., b] = abs(u * c) + abs(w * s), abs(w * c) + abs(u * s)
    return y, mag


def quantise(x: np.ndarray, group: int):
    """(codes uint8 [..][dim], pairs fp16 [..][dim / group][2] of step and offset) of fp32 rows."""
    g = x.astype(np.float32).reshape(x.shape[:-1] + (-1, group))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        bad = ~np.isfinite(g).all(-1)
        low, high = g.min(-1), g.max(-1)
        m, s = low.astype(np.float16), ((high - low) / np.float32(15)).astype(np.float16)
        bad |= ~np.isfinite(m)
        m, s = np.where(bad, np.float16(np.nan), m), np.where(bad, np.float16(0), s)
        c = np.rint((g - m[..., None].astype(np.float32)) / s[..., None].astype(np.float32))
        c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0)
    return np.nan_to_num(c).astype(np.uint8).reshape(x.shape), np.stack([s, m], axis=-1)


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def value_f64(packed: np.ndarray, pairs: np.ndarray) -> np.ndarray:
    """What code bytes [..][dim / 2] with their pairs stand for."""
    c = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), dtype=np.float64)
    c[..., 0::2], c[..., 1::2] = packed & 15, packed >> 4
    group = c.shape[-1] // pairs.shape[-2]
    p = np.repeat(pairs.astype(np.float64), group, axis=-2)
    return p[..., 1] + p[..., 0] * c


def bounds(keys: np.ndarray) -> np.ndarray:
    """Least and greatest key per column of every block of 64 tokens, [blocks][heads][2][dim], from fp16 keys [n][heads][dim]."""
    return np.stack([np.stack([b.min(0), b.max(0)], axis=1) for b in
                     (keys[i: i + 64] for i in range(0, len(keys), 64))])
