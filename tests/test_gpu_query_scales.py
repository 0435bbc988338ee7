"""GPU: paged_query_attention over FP8 pools whose blocks' value scales lie many powers of two apart: a row's result
depends on the scales that it sees alone, and on those as far as its weights reach them.

Tolerance, row by row and element by element (p the softmax weights, s_j the value scale of key j, |code| <= 448).  A weight's
relative error e_j: the float32 product sum, (d + 8) 2^-23 of |q||k| scale; the roundings of t_j and of its distance to the
base, 2^-22 of their sizes (the base is moved by log2 of a scale, at most 40, and 8); the exponential, 2^-22; sums over n
keys, (n/16 + 64) 2^-23.  It moves the row by sum p_j e_j |v_j| and, through the sum of weights, by |out| sum p_j e_j.
p_j s_j enters the products as float16: 2^-11 of itself, or 2^-25 where the largest is 2^7 or more, n 2^-32 of it in all.
The result is rounded once."""

import math

import numpy as np
import pytest
import torch

import test_gpu_query as G
from oracle import query as OQ

pytestmark = pytest.mark.gpu


def within(got, want, tol, what):
    """want - tol <= got <= want + tol, where a bound beyond float16's largest value, 65504, may come as that value or as
    infinity: x in [lo, hi] rounds to float16 between lo and hi rounded, and what is beyond 65504 rounds to either of them.
    (A sum of scales of 2^30 may cancel to less than its error, so that even its sign is open.)"""
    lo, hi = want - tol, want + tol
    fine = (got >= np.where(lo < -65504, -np.inf, np.minimum(lo, 65504))) & (got <= np.where(hi > 65504, np.inf, np.maximum(hi, -65504)))
    assert fine.all(), (what, float(np.max(np.abs(got - want)[~fine] / tol[~fine])))


def row_close(b, s, q, i, n, got, sl, window, rng, scale, what):
    k, v = b.values(s, "k"), b.values(s, "v")
    c, d = b.lens[s], b.d
    p = c - n + i
    lo, hi = OQ.visible(n, c, i, window, rng)
    if lo == hi:
        assert not got.any()
        return
    want = OQ.query_attention(q[None], k[:p + 1], v[:p + 1], scale, 0, 0.0, sl, np.array([[lo, hi]])) if hi <= p + 1 else None
    t = OQ.scores(q, k[lo:hi], p, lo, scale, 0.0, sl)                  # [Hq, m]
    w = np.exp(t - t.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    group = q.shape[0] // b.H
    sc = b.vs[b.tab[s][np.arange(lo, hi) // b.B]].astype(np.float64)
    for h in range(q.shape[0]):
        vv, qq = v[lo:hi, h // group], q[h].astype(np.float64)
        m = hi - lo
        out = w[h] @ vv
        if want is not None:
            assert np.allclose(out, want[0, h], rtol=1e-9, atol=1e-12 * float(np.max(w[h] @ np.abs(vv))))
        mag = np.linalg.norm(qq) * np.linalg.norm(k[lo:hi, h // group], axis=-1) * scale
        e = (d + 8) * 2.0 ** -23 * mag + 2.0 ** -22 * (np.abs(t[h]) + np.abs(t[h]).min() + 50) + 2.0 ** -22 + (m / 16 + 64) * 2.0 ** -23
        a = (w[h] * e) @ np.abs(vv) + np.abs(out) * (w[h] @ e)
        tol = a + 2.0 ** -11 * (w[h] @ np.abs(vv)) + m * 2.0 ** -32 * 448 * np.max(w[h] * sc) + 2.0 ** -11 * np.abs(out) + 2.0 ** -25
        within(got[h], out, tol, (what, s, i, h))


def check(b, new, group, ranges=None, slopes=None, window=0, what=None):
    rng, Hq, scale = b.rng, b.H * group, 1 / math.sqrt(b.d)
    q = rng.standard_normal((sum(new), Hq, b.d)).astype(np.float16)
    start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    up = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=t))).cuda()       # noqa: E731
    got = b.cache.query_attention(0, torch.from_numpy(q).cuda(), up(start), up(b.tab), up(b.lens), max(new), max(b.lens), scale,
                                  window=window, slopes=None if slopes is None else up(slopes, np.float32),
                                  ranges=None if ranges is None else up(ranges)).cpu().numpy().astype(np.float64)
    assert b.cache.device_error() == 0
    for s, n in enumerate(new):
        for i in range(n) if n <= 40 else sorted(set(range(0, n, 7)) | {n - 1}):
            r = start[s] + i
            row_close(b, s, q[r], i, n, got[r], slopes, window, None if ranges is None else ranges[r], scale, what)


def scaled(d, H, B, lens, of, seed=0):
    """A batch whose block j of a sequence (of nb) has the value scale of(j, nb)."""
    b = G.Batch("fp8", d, H, B, lens, seed=seed)
    for s, c in enumerate(b.lens):
        nb = -(-c // B)
        for j in range(nb):
            b.vs[b.tab[s][j]] = of(j, nb)
    b.upload()
    return b


@pytest.mark.parametrize("new", [[300, 130], [1, 4]])
@pytest.mark.parametrize("power", [10, 20, 34, 50])
def test_documents_beside_larger_scales(power, new):
    """Documents of 64 positions whose scales are 2^-4 and 2^(power - 4) in turn, each row seeing its own only."""
    lens = [420, 200]
    b = scaled(128, 2, 16, lens, lambda j, nb: 2.0 ** (-4 + power * (j // 4 % 2)))
    p = np.concatenate([np.arange(c - n, c) for n, c in zip(new, lens)])
    check(b, new, 2, ranges=np.stack((p // 64 * 64, p + 1), 1), what=power)
    # the same rows in the other order of scales
    b2 = scaled(128, 2, 16, lens, lambda j, nb: 2.0 ** (-4 + power * (1 - j // 4 % 2)), seed=1)
    check(b2, new, 2, ranges=np.stack((p // 64 * 64, p + 1), 1), what=power)
    b.cache.close()
    b2.cache.close()


@pytest.mark.parametrize("new", [[260, 100], [2, 3]])
@pytest.mark.parametrize("power", [20, 45])
def test_rows_before_a_larger_scale(power, new):
    """Causal rows; the last block's scale is 2^power times the others'."""
    b = scaled(64, 2, 8, [263, 102], lambda j, nb: 2.0 ** (-6 + (power if j == nb - 1 else 0)))
    check(b, new, 1, what=power)
    b.cache.close()


@pytest.mark.parametrize("new", [[200, 77], [1, 5]])
@pytest.mark.parametrize("far", [20, 38, 60, 100])
def test_large_scales_far_away(far, new):
    """Blocks of large scales that the distance bias leaves next to no weight: the near ones decide, or both."""
    b = scaled(128, 2, 16, [400, 150], lambda j, nb: 2.0 ** (-3 + (far if j < nb // 2 else 0)))
    sl = np.array([3.0, 0.5, 0.2, 0.05], dtype=np.float32)
    check(b, new, 2, slopes=sl, what=far)
    b.cache.close()


@pytest.mark.parametrize("new", [[200, 77], [1, 5]])
def test_falling_and_rising_scales(new):
    """Every block's scale a step of 2^3 from the last one's, down and up, from 2^-40 to 2^8; zeros among them; a window."""
    for of in (lambda j, nb: 2.0 ** (8 - 3 * (j % 16)), lambda j, nb: 2.0 ** (-40 + 3 * (j % 16)),
               lambda j, nb: 0.0 if j % 3 else 2.0 ** (-30 + 2 * (j % 16))):
        b = scaled(128, 1, 8, [333, 140], of)
        check(b, new, 4, what="all")
        check(b, new, 4, window=20, what="window")
        b.cache.close()


@pytest.mark.parametrize("d,group", [(128, 8), (64, 1)])
def test_parts_of_different_scales(d, group):
    """Contexts cut into parts (of CTAs, and of keys), with scales that differ from part to part."""
    for new, lens in (([40], [4000]), ([2], [9000])):
        b = scaled(d, 1, 16, lens, lambda j, nb: 2.0 ** (-8 + 30 * (j // 32 % 2)), seed=d)
        p = np.arange(lens[0] - new[0], lens[0])
        check(b, new, group, what="all")
        # rows that see a large and a small part only
        r = np.stack((np.zeros_like(p), np.where(p % 2, 512, 400)), 1)
        r[1::3] = (512, 1024)
        check(b, new, group, ranges=r, what="ranges")
        b.cache.close()


@pytest.mark.parametrize("new", [[150, 60], [1, 3]])
@pytest.mark.parametrize("odd", [-0.01, -300.0, 2.0 ** 25, 2.0 ** 100, math.inf, -math.inf, math.nan])
def test_scales_that_are_none(odd, new):
    """Blocks whose value scale is negative, enormous or not finite: as the definition has them for rows that see them, and
    nothing to rows that do not."""
    lens = [200, 90]
    b = scaled(128, 2, 16, lens, lambda j, nb: odd if j == nb - 3 else 0.01)
    p = np.concatenate([np.arange(c - n, c) for n, c in zip(new, lens)])
    first = np.concatenate([np.full(n, (-(-c // 16) - 2) * 16) for n, c in zip(new, lens)])
    # every other row begins behind those blocks, where it stands behind them itself; rows before them do not reach them
    r = np.stack((np.where((np.arange(len(p)) % 2 == 0) & (p >= first), first, 0), p + 1), 1)
    if math.isfinite(odd):
        check(b, new, 2, ranges=r, what=odd)
    else:
        seen = np.concatenate([(r[:new[0], 0] < first[0]) & (p[:new[0]] >= first[0] - 16),
                               (r[new[0]:, 0] < first[-1]) & (p[new[0]:] >= first[-1] - 16)])
        Hq, scale = 4, 1 / math.sqrt(128)
        q = b.rng.standard_normal((sum(new), Hq, 128)).astype(np.float16)
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        up = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=t))).cuda()       # noqa: E731
        got = b.cache.query_attention(0, torch.from_numpy(q).cuda(), up(start), up(b.tab), up(lens), max(new), max(lens), scale,
                                      ranges=up(r)).cpu().numpy().astype(np.float64)
        assert b.cache.device_error() == 0 and seen.any() and not seen.all()
        for s, n in enumerate(new):
            b.vs[b.tab[s][-(-lens[s] // 16) - 3]] = 0.01       # (the values of rows that do not see it)
            for i in range(n):
                at = start[s] + i
                if seen[at]:
                    assert not np.isfinite(got[at]).any(), (s, i)
                else:
                    row_close(b, s, q[at], i, n, got[at], None, 0, r[at], scale, odd)
    b.cache.close()
