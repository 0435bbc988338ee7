"""GPU: how exact 4-bit decode attention is, over the whole range of scores, queries and scales.

Tolerance, derived: with weights p_t and values v_t the result is sum p v / sum p, so a relative
error e in every weight moves it by at most 2 e max|v|.  A score is a float32 sum of exact products
(K values and queries are float16, and are used as they are): 136 additions, each off by at most
2^-23 of sum |q||k|.  The weight is 2^x with x the score's distance from the base times scale
log2(e), at most 15 above it: 15 roundings of 2^-24 for the product, 2^-23 more for the factor,
2^-22 for the exponential; and it enters the products as two float16 terms, off by 2^-22.  Sums over
n tokens are float32: one rounding per 16 tokens and part, counted as (n/16 + 40) 2^-24."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import int4 as O4
from paged_kv_cache_169_gb300.cache import PagedKVCache

pytestmark = pytest.mark.gpu


def run(k, v, q, B, scale, **more):
    """k, v: (codes, scale bytes) [n, H, d] of one sequence, q float16 [Hq, d].  The kernel's result and
    the float64 one, with the tolerance."""
    n, H, d = k[0].shape
    nb = -(-n // B)
    cache = PagedKVCache(1, nb, B, H, d, "int4")
    tab = np.random.default_rng(n).permutation(nb).astype(np.int32)
    for t, which, (c, s) in ((cache.k[0], "k", k), (cache.v[0], "v", v)):
        p = np.zeros(tuple(t.shape), dtype=np.uint8)
        for i in range(n):
            for h in range(H):
                O4.store(p, which, tab[i // B], h, i % B, c[i, h], s[i, h])
        t.copy_(torch.from_numpy(p))
    got = cache.attention_ex(0, torch.from_numpy(q[None]).cuda(), torch.from_numpy(tab[None]).cuda(),
                             torch.tensor([n], dtype=torch.int32, device="cuda"), n, scale, **more)
    assert cache.device_error() == 0
    cache.close()
    kx, vx = O4.dequantize(*k), O4.dequantize(*v)
    G = q.shape[0] // H
    want, tol = np.zeros(q.shape), np.zeros((q.shape[0], 1))
    for j in range(q.shape[0]):
        qj = q[j].astype(np.float64)
        want[j] = OA.decode_attention_one(qj, kx[:, j // G], vx[:, j // G], scale)
        mag = np.max(np.abs(kx[:, j // G]) @ np.abs(qj)) * scale
        e = 136 * 2.0 ** -23 * mag + 45 * 2.0 ** -24 + 2.0 ** -21 + (n / 16 + 40) * 2.0 ** -24
        tol[j] = 2 * e * np.max(np.abs(vx))
    return got[0].double().cpu().numpy(), want, tol


def random_tokens(rng, n, H, d, lo=80, hi=110):
    return (rng.integers(-7, 8, (n, H, d)).astype(np.int8),
            rng.integers(lo, hi, (n, H, d // 16)).astype(np.uint8))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d,n", [(128, 3), (128, 100), (64, 5), (64, 700)])
def test_weights_are_not_rounded_to_float16(G, d, n):
    """Small scores, so that every token counts and the error of the weights shows."""
    rng = np.random.default_rng(G * n)
    q = (rng.standard_normal((2 * G, d)) * 0.02).astype(np.float16)
    got, want, tol = run(random_tokens(rng, n, 2, d), random_tokens(rng, n, 2, d), q, 16, 1 / math.sqrt(d))
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


def one_hot_tokens(n, d, at, low):
    """n tokens of one head: `low` (code, scale byte) in element 0, but for tokens in `at`: {token:
    [(element, code, scale byte)]}."""
    c, s = np.zeros((n, 1, d), dtype=np.int8), np.zeros((n, 1, d // 16), dtype=np.uint8)
    for t in range(n):
        for e, code, byte in at.get(t, [(0, *low)]):
            c[t, 0, e], s[t, 0, e // 16] = code, byte
    return c, s


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_whose_float32_step_is_as_large_as_the_slack(G, d):
    """Two sums of products, 349440000 and 349440064 (every sum exact in float32, where neighbours are 32
    apart), in different chunks: weights of 0.0035 and 0.9965 at scale 1/sqrt(128).  The scores' distances
    are exact, so the sums' error does not enter the tolerance."""
    rng = np.random.default_rng(d + G)
    n, byte832, byte16 = 130, O4.encode_scale(832.0), O4.encode_scale(16.0)
    k = one_hot_tokens(n, d, {3: [(0, 7, byte832)], 100: [(0, 7, byte832), (18, 4, byte16)]}, (-7, byte832))
    v = random_tokens(rng, n, 1, d)
    q = np.zeros((G, d), dtype=np.float16)
    q[:, 0], q[:, 18] = 60000, 1
    kx = O4.dequantize(*k)[:, 0]
    assert sorted(set(kx @ q[0].astype(np.float64)))[-2:] == [349440000.0, 349440064.0]
    for scale in (1 / math.sqrt(128), 0.01, 0.5):
        got, want, _ = run(k, v, q, 16, scale)
        tol = 2 * (45 * 2.0 ** -24 + 2.0 ** -21 + 60 * 2.0 ** -24) * np.max(np.abs(O4.dequantize(*v)))
        assert np.all(np.abs(got - want) <= tol), (scale, np.max(np.abs(got - want)), tol)


@pytest.mark.parametrize("partition", [0, 32])
@pytest.mark.parametrize("G,d", [(1, 128), (8, 128), (4, 64)])
def test_scales_up_to_the_largest(G, d, partition):
    """With scores of 10^30 and more apart one token has all the weight: its values, exactly.  In one
    range and in parts that warps and CTAs join."""
    rng = np.random.default_rng(d)
    n = 2000
    k, v = random_tokens(rng, n, 1, d), random_tokens(rng, n, 1, d)
    q = rng.integers(-9, 10, (G, d)).astype(np.float16)
    kx, vx = O4.dequantize(*k)[:, 0], O4.dequantize(*v)[:, 0]
    best = np.argmax(kx @ q.astype(np.float64).T, axis=0)
    for scale in (1e20, 1e30, 1e37, 2.9e38):
        got, _, _ = run(k, v, q, 16, scale, partition_tokens=partition)
        assert np.array_equal(got, vx[best]), scale


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [0, 1])
def test_small_queries_keep_their_bits(G, d, odd):
    """Queries down to the smallest float16, in even and in odd elements, beside keys and a scale that
    make them count."""
    rng = np.random.default_rng(d + G + odd)
    n = 90
    q = np.zeros((G, d), dtype=np.float16)
    q[:, odd::2] = rng.integers(-40, 41, (G, d // 2)) * 2.0 ** -24
    k, v = random_tokens(rng, n, 1, d, 184, 199), random_tokens(rng, n, 1, d)
    got, want, tol = run(k, v, q, 8, 2.0)
    assert np.ptp(O4.dequantize(*k)[:, 0] @ q[0].astype(np.float64)) * 2 > 0.05          # the scores do differ
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
