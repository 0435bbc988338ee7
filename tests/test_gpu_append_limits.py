"""GPU: the fused append at the edges of what it may store."""

import numpy as np
import pytest
import torch

from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache

pytestmark = pytest.mark.gpu


def lengths_too_long(pool, G, d, B, **more):
    """A sequence whose length is beyond max_context, or beyond its table row, or negative, has no
    place for a new token: KV_DEVERR_CONTEXT, nothing stored, and the attention over its clamped length
    is that of the cache as it was.  Its neighbours' tokens are stored."""
    rng = np.random.default_rng(d + B + G)
    H, limit, width = 2, 3 * B + 5, 4
    nb = 5 * width
    cache = PagedKVCache(1, nb, B, H, d, pool)
    dt = torch.float32 if pool == "f32" else torch.float16
    for t in cache.k + cache.v:
        if pool == "int4":
            a = rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)
            a[..., 4 * d:] = rng.integers(80, 110, a[..., 4 * d:].shape)
            t.copy_(torch.from_numpy(a))
        elif pool == "fp8":
            t.copy_(torch.from_numpy(rng.integers(0, 120, tuple(t.shape), dtype=np.uint8)))
        else:
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
    tab = torch.from_numpy(rng.permutation(nb).astype(np.int32).reshape(5, width)).cuda()
    q = torch.from_numpy(rng.standard_normal((5, H * G, d)).astype(np.float32)).cuda().to(dt)
    kn, vn = (torch.from_numpy(rng.standard_normal((5, H, d)).astype(np.float32)).cuda().to(dt) for _ in range(2))
    full = width * B                                   # what a table row holds
    for limit in (limit, full, full + 7):
        most = min(limit, full)
        lens = torch.tensor([most, most + 1, 9, -3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        clamped = torch.tensor([most, most, 9, 0, most], dtype=torch.int32, device="cuda")
        good = [0, 2]
        before = [cache.k[0].clone(), cache.v[0].clone()]
        plain = cache.attention_ex(0, q, tab, clamped, limit, 0.1, **more).clone()
        assert cache.device_error() == 0
        out = cache.attention_ex(0, q, tab, lens, limit, 0.1, k_new=kn, v_new=vn, **more)
        assert cache.device_error() == abi.KV_DEVERR_CONTEXT
        after = [cache.k[0].clone(), cache.v[0].clone()]
        for old, new in zip(before, after):
            changed = set((old != new).flatten(1).any(1).nonzero().flatten().tolist())
            assert changed == {int(tab[s, (int(clamped[s]) - 1) // B]) for s in good}
        for s in (1, 3, 4):
            assert torch.equal(out[s], plain[s]), s
        want = cache.attention_ex(0, q, tab, clamped, limit, 0.1, **more)
        for s in good:                                 # as after a separate append
            assert torch.equal(out[s], want[s]), s
        for t, old in zip((cache.k[0], cache.v[0]), before):
            t.copy_(old)
    assert cache.device_error() == 0
    cache.close()


@pytest.mark.parametrize("G,d,B", [(1, 128, 16), (4, 64, 8), (8, 128, 32)])
def test_int4_lengths_too_long_store_nothing(G, d, B):
    lengths_too_long("int4", G, d, B)
    lengths_too_long("int4", G, d, B, window=20)
    lengths_too_long("int4", G, d, B, partition_tokens=32)


@pytest.mark.parametrize("pool,G,d,B", [("f32", 1, 128, 16), ("f32", 1, 64, 8), ("f16", 1, 128, 16), ("f16", 1, 64, 32),
                                        ("f16", 4, 128, 16), ("f16", 8, 128, 8), ("f16", 2, 64, 16),
                                        ("fp8", 1, 128, 16), ("fp8", 1, 64, 8), ("fp8", 8, 128, 32), ("fp8", 4, 64, 16)])
def test_lengths_too_long_store_nothing(pool, G, d, B):
    lengths_too_long(pool, G, d, B)
    lengths_too_long(pool, G, d, B, window=20)
    lengths_too_long(pool, G, d, B, partition_tokens=32, flags=abi.KV_DECODE_PDL | abi.KV_DECODE_EARLY_TABLES)


@pytest.mark.parametrize("pool,G,d,B", [("f32", 1, 128, 16), ("f16", 1, 128, 16), ("f16", 1, 64, 32), ("f16", 4, 128, 16),
                                        ("f16", 2, 64, 16), ("fp8", 1, 128, 16), ("fp8", 8, 128, 32), ("fp8", 1, 64, 8),
                                        ("int4", 1, 128, 16), ("int4", 8, 64, 8)])
def test_bad_block_ids_store_nothing(pool, G, d, B):
    """A new token whose block id lies outside the pool is stored nowhere (block 0, which is read in its
    place, belongs to another sequence); a sequence whose token goes into block 0 has it stored."""
    rng = np.random.default_rng(d + B + G)
    H, nb = 2, 9
    cache = PagedKVCache(1, nb, B, H, d, pool)
    dt = torch.float32 if pool == "f32" else torch.float16
    for t in cache.k + cache.v:
        if t.dtype == torch.uint8:
            t.copy_(torch.from_numpy(rng.integers(80, 110, tuple(t.shape), dtype=np.uint8)))
        else:
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
    tab = np.array([[3, 4, -5], [1, nb, -1], [2, 0, -1], [5, 2 ** 31 - 1, 6]], dtype=np.int32)
    lens = torch.tensor([2 * B + 1, B + 3, 2 * B, B + 1], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((4, H * G, d)).astype(np.float32)).cuda().to(dt)
    kn, vn = (torch.from_numpy(rng.standard_normal((4, H, d)).astype(np.float32)).cuda().to(dt) for _ in range(2))
    before = [cache.k[0].clone(), cache.v[0].clone()]
    cache.attention_ex(0, q, torch.from_numpy(tab).cuda(), lens, 3 * B, 0.1, k_new=kn, v_new=vn)
    assert cache.device_error() == abi.KV_DEVERR_BLOCK_ID
    slots = torch.tensor([-1, -1, B - 1, -1], device="cuda")           # block 0, its last row
    fused = [cache.k[0].clone(), cache.v[0].clone()]
    for t, old in zip((cache.k[0], cache.v[0]), before):
        t.copy_(old)
    cache.append(0, kn, vn, slots)
    assert torch.equal(fused[0], cache.k[0]) and torch.equal(fused[1], cache.v[0])
    cache.close()
