"""GPU: paged_query_attention with caps of any size.  A cap far above the scores leaves them as they are; the error of a
capped score is a part of the score, not of the cap.

Oracle and tolerance: test_gpu_query's, with the cap's term 2^-20 of the smaller of the cap and the largest score (above a cap
of 64 the series or the exponential form of tanh is within 2^-21 of the score, and the multiplications before it within
2^-22; up to 64, 2^-20 of the cap, which is 2^-14 at most)."""

import math

import numpy as np
import pytest
import torch

import test_gpu_query as G
from oracle import query as OQ

pytestmark = pytest.mark.gpu


def up(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).cuda()


def check(b, new, group, cap, qmul=1.0, slopes=None):
    Hq, scale = b.H * group, 1 / math.sqrt(b.d)
    q = (b.rng.standard_normal((sum(new), Hq, b.d)) * qmul).astype(np.float32 if b.pool == "f32" else np.float16)
    start = np.concatenate(([0], np.cumsum(new)))
    got = b.cache.query_attention(0, torch.from_numpy(q).cuda(), up(start), up(b.tab), up(b.lens), max(new), max(b.lens), scale,
                                  score_cap=cap, slopes=None if slopes is None else up(slopes, np.float32)).cpu().numpy()
    assert b.cache.device_error() == 0
    for s, n in enumerate(new):
        rows = slice(start[s], start[s + 1])
        k, v = b.values(s, "k"), b.values(s, "v")
        want = OQ.query_attention(q[rows], k, v, scale, 0, cap, slopes)
        x_max = float(np.max(np.linalg.norm(q[rows].astype(np.float64), axis=-1)) * np.max(np.linalg.norm(k, axis=-1))) * scale
        t_max = min(cap, x_max) + (b.lens[s] * float(np.max(slopes)) if slopes is not None else 0.0)
        small = cap if cap <= 64 else min(cap, x_max)
        tol = G.tolerance(b.pool, q[rows].astype(np.float64), k, v, t_max, scale, small, want)
        G.close(got[rows], want, tol, (cap, s, n))


@pytest.mark.parametrize("pool", G.POOLS)
@pytest.mark.parametrize("cap", [2.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e10, 1e30, 2.9e38])
@pytest.mark.parametrize("new", [[130, 40], [1, 4]])
def test_caps_of_any_size(pool, cap, new):
    b = G.Batch(pool, 128, 2, 16, [333, 150], seed=3)
    check(b, new, 2, cap)
    check(b, new, 2, cap, slopes=np.array([0.3, 0.1, 0.02, 0.5], dtype=np.float32))
    b.cache.close()


@pytest.mark.parametrize("pool", G.POOLS)
@pytest.mark.parametrize("new", [[200], [3]])
def test_scores_near_and_above_a_large_cap(pool, new):
    """Scores from far below half the cap, where the series ends, to far above the cap."""
    b = G.Batch(pool, 64, 1, 8, [300], seed=5)
    for cap, qmul in ((80.0, 16.0), (200.0, 30.0), (70.0, 200.0), (1000.0, 500.0)):
        check(b, new, 4, cap, qmul)
    b.cache.close()


@pytest.mark.parametrize("new", [[60], [2]])
def test_parts_with_a_large_cap(new):
    b = G.Batch("f16", 128, 1, 16, [6000], seed=6)
    check(b, new, 2, 1e6)
    check(b, new, 2, 1e3, qmul=8.0)
    b.cache.close()
