"""Oracle: attention of a sequence's newest tokens over its cached context (test infrastructure only).

[KV Cache篇] §3.1 adds a mask to the scores of the new tokens over ``cache[:start_pos + seqlen]``
before the softmax.  Row i of n new tokens over c cached ones stands at p = c - n + i and sees the
positions first <= j < end (0 and p + 1, or the row's own range) with p - j < window; its scores are

    t_j = cap tanh(x_j / cap) - slope |p - j|,   x_j = scale q_i . k_j

and its result is sum_j softmax(t)_j v_j over what it sees, 0 where that is nothing.
"""

from __future__ import annotations

import numpy as np


def visible(n: int, c: int, i: int, window: int = 0, rng=None) -> tuple[int, int]:
    """[first, end) of the positions row i sees; (0, 0) for none."""
    p = c - n + i
    first, end = (0, p + 1) if rng is None else (int(rng[0]), int(rng[1]))
    if window > 0:
        first = max(first, p - window + 1)
    first, end = max(first, 0), min(end, c)
    return (first, end) if first < end else (0, 0)


def scores(q, k, p: int, first: int, scale: float, cap: float = 0.0, slopes=None) -> np.ndarray:
    """float64 [Hq, m] for q [Hq, d] at position p over k [m, H, d] at positions first, first + 1, ..."""
    q, k = np.asarray(q, dtype=np.float64), np.asarray(k, dtype=np.float64)
    group = q.shape[0] // k.shape[1]
    x = np.stack([k[:, h // group] @ q[h] for h in range(q.shape[0])]) * scale
    if cap > 0:
        x = cap * np.tanh(x / cap)
    if slopes is not None:
        x = x - np.asarray(slopes, dtype=np.float64)[:, None] * np.abs(p - (first + np.arange(k.shape[0])))
    return x


def query_attention(q, k, v, scale: float, window: int = 0, cap: float = 0.0, slopes=None,
                    ranges=None) -> np.ndarray:
    """q [n, Hq, d], k and v [c, H, d], ranges None or [n, 2].  Returns float64 [n, Hq, d]."""
    n, hq, d = np.asarray(q).shape
    c = np.asarray(k).shape[0]
    out = np.zeros((n, hq, d))
    for i in range(n):
        lo, hi = visible(n, c, i, window, None if ranges is None else ranges[i])
        if lo == hi:
            continue
        t = scores(q[i], k[lo:hi], c - n + i, lo, scale, cap, slopes)
        w = np.exp(t - t.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        vv = np.asarray(v[lo:hi], dtype=np.float64)
        group = hq // vv.shape[1]
        for h in range(hq):
            out[i, h] = w[h] @ vv[:, h // group]
    return out
