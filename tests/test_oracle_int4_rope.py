"""Pins of the 4-bit and rotation oracles (CPU): closed forms and round trips."""

import math

import numpy as np
import pytest

from oracle import int4 as O4
from oracle import rope as OR


def test_scale_bytes_are_float16_bits():
    b = np.arange(256, dtype=np.uint16)
    want = (b << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(O4.SCALES, want, equal_nan=True)


def test_encode_scale_is_nearest_even():
    for b in range(O4.encode_scale(896.0) + 1):
        assert O4.encode_scale(O4.SCALES[b]) == b
    for b in range(O4.encode_scale(896.0)):
        mid = (O4.SCALES[b] + O4.SCALES[b + 1]) / 2
        assert O4.encode_scale(mid) == b + b % 2
        assert O4.encode_scale(np.nextafter(mid, 0)) == b
        assert O4.encode_scale(np.nextafter(mid, 1e9)) == b + 1
    assert O4.decode_scale(O4.encode_scale(1e9)) == 896.0


@pytest.mark.parametrize("d", [64, 128])
def test_quantize_error_bound(d):
    """A value is off by at most half a scale, plus what a scale rounded down clips from the top:
    amax <= 7 s (1 + 2^-4), so at most 7/16 of a scale."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((200, d)) * np.exp2(rng.uniform(-6, 6, (200, 1)))).astype(np.float16)
    c, s = O4.quantize(x)
    err = np.abs(O4.dequantize(c, s) - x.astype(np.float64)).reshape(200, -1, 16)
    assert np.all(err <= 0.5 * O4.SCALES[s][..., None] * (1 + 1e-6))
    assert c.min() >= -7 and c.max() <= 7


def test_quantize_special_groups():
    x = np.zeros((5, 16), dtype=np.float32)
    x[1, 3] = np.nan
    x[2, 0], x[2, 1] = np.inf, -1e30
    x[3, 5] = 7e5
    x[4] = 1e-8
    c, s = O4.quantize(x)
    v = O4.dequantize(c, s)
    assert np.all(v[0] == 0) and np.all(np.isnan(v[1]))
    assert v[2, 0] == 6272 and v[2, 1] == -6272 and np.all(v[2, 2:] == 0)
    assert v[3, 5] == 6272 and np.all(v[4] == 0)


@pytest.mark.parametrize("d,B", [(64, 8), (128, 16), (128, 32), (64, 32)])
def test_layout_round_trip_and_bijection(d, B):
    rng = np.random.default_rng(2)
    for which in "kv":
        pool = rng.integers(0, 256, (3, 2, B // 8, 4 * d + d // 2), dtype=np.uint8)
        before = pool.copy()
        want = {}
        for b in range(3):
            for h in range(2):
                for off in range(B):
                    c = rng.integers(-7, 8, d).astype(np.int8)
                    s = rng.integers(0, 200, d // 16).astype(np.uint8)
                    O4.store(pool, which, b, h, off, c, s)
                    want[b, h, off] = (c, s)
        for (b, h, off), (c, s) in want.items():
            c2, s2 = O4.load(pool, which, b, h, off, d)
            assert np.array_equal(c, c2) and np.array_equal(s, s2)
        # every byte of the pool belongs to exactly one token: the originals are all gone
        assert (pool != before).mean() > 0.9
        blk, off = np.array([2, 0, 1]), np.array([B - 1, 3, 6])
        got = O4.token_values(pool, which, d, blk, off)
        for i in range(3):
            for h in range(2):
                c, s = want[int(blk[i]), h, int(off[i])]
                assert np.array_equal(got[i, h], O4.dequantize(c, s))


def test_rotation_closed_forms():
    t = OR.table(50, 32, 10000.0)
    assert np.all(t[0, :16] == 1) and np.all(t[0, 16:] == 0)
    assert math.isclose(t[7, 16 + 3], math.sin(7 * 10000.0 ** (-6 / 32)), rel_tol=1e-14)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 2, 64))
    for adjacent in (False, True):
        y = OR.rotate(x, t, 32, adjacent)
        assert np.array_equal(y[..., 32:], x[..., 32:])               # not rotated
        assert np.array_equal(y[0], x[0])                             # position 0
        assert np.allclose(np.sum(y ** 2, -1), np.sum(x ** 2, -1))    # a rotation keeps lengths
        back = OR.rotate(y, np.concatenate([t[:, :16], -t[:, 16:]], 1), 32, adjacent)
        assert np.allclose(back, x, atol=1e-14)
        # scores depend on the distance of positions only
        q, k = np.broadcast_to(x[1], x.shape), np.broadcast_to(x[2], x.shape)
        s = np.einsum("nhd,nhd->nh", OR.rotate(q, t, 32, adjacent)[5:], OR.rotate(k, t, 32, adjacent)[:-5])
        assert np.allclose(s, s[:1])
    assert not np.allclose(OR.rotate(x, t, 32, False)[1:], OR.rotate(x, t, 32, True)[1:])
