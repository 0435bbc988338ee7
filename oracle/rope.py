"""Oracle: rotation of queries and keys by position (test infrastructure only).

[KV Cache篇] §3.1 applies ``apply_rotary_emb`` to the projections before the cache write.  Pair i
of a head's first R elements, (x, y), is turned by the angle ``a = p * base**(-2i/R)`` at
position p:

    x' = x cos a - y sin a,    y' = y cos a + x sin a

Pairs are elements (i, i + R/2) ("half") or (2i, 2i + 1) ("adjacent"); the rest of the head is
unchanged.
"""

from __future__ import annotations

import math

import numpy as np


def angle(position: int, i: int, rot_dim: int, base: float) -> float:
    return position * math.pow(base, -2.0 * i / rot_dim)


def table(positions: int, rot_dim: int, base: float) -> np.ndarray:
    """float64 [positions, rot_dim]: cosines, then sines."""
    f = np.array([math.pow(base, -2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    a = np.arange(positions, dtype=np.float64)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x, cos_sin_rows, rot_dim: int, adjacent: bool, dtype=np.float64) -> np.ndarray:
    """x [n, heads, d], cos_sin_rows [n, rot_dim] (each token's row).  Every product and sum is
    rounded to ``dtype`` on its own."""
    y = np.array(x, dtype=dtype)
    row = np.asarray(cos_sin_rows, dtype=dtype)[:, None]
    half = rot_dim // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        u, w = y[..., a].copy(), y[..., b].copy()
        c, s = row[..., i], row[..., half + i]
        y[..., a] = u * c - w * s
        y[..., b] = w * c + u * s
    return y
