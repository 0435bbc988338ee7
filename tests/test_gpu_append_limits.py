"""GPU: the fused append at the edges of what it may store."""

import numpy as np
import pytest
import torch

from oracle import int4 as O4
from oracle import rope as OR
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_table

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


@pytest.mark.parametrize("in_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("d,B", [(128, 16), (64, 8)])
def test_a_group_with_a_nan_is_the_same_bytes_from_every_call(in_dtype, d, B):
    """kv_append, kv_append_rope and the fused decode step, neighbours in one V word or not: the scale
    byte of a NaN and codes of 0."""
    rng = np.random.default_rng(d)
    H, n = 2, 24
    x = rng.standard_normal((2, n, H, d)).astype(np.float32)
    x[:, 1, 0, 3] = x[:, 2, 1, 17] = x[:, 3, 0, d - 1] = x[:, 8, 1, 0] = np.nan
    x[:, 5, 0, 16:32] = np.nan
    x[:, 6, 0, 4], x[:, 6, 0, 5] = np.nan, np.inf
    x[:, 11, 1, 9] = np.array([0xFFC01234], dtype=np.uint32).view(np.float32)[0]         # a NaN of another sign
    k, v = (torch.from_numpy(a).cuda().to(in_dtype) for a in x)
    # half of the tokens side by side, the others anywhere; the fused call, whose sequences share no
    # block, puts token i into block i
    slots = np.concatenate([np.arange(12) + n, rng.permutation(n)[:12]]).astype(np.int64)
    alone = (np.arange(n) * B + rng.integers(0, B, n)).astype(np.int64)
    caches = [PagedKVCache(1, n, B, H, d, "int4") for _ in range(3)]
    for c in caches:
        c.k[0].zero_()
        c.v[0].zero_()
    caches[0].append(0, k, v, torch.from_numpy(slots).cuda())
    caches[1].append_rope(0, k, v, torch.from_numpy(slots).cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"),
                          rope_table(1, d))
    q = torch.zeros(n, H, d, device="cuda").half()
    t = torch.from_numpy(alone).cuda()
    caches[2].attention_ex(0, q, (t // B).to(torch.int32).reshape(n, 1), (t % B + 1).to(torch.int32), B, 0.1,
                           k_new=k, v_new=v)
    # at position 0 a key's pairs turn by nothing, but a NaN or an infinity times 0 makes its partner a NaN
    with np.errstate(invalid="ignore"):
        turned = OR.rotate(k.cpu().numpy(), rope_table(1, d).cpu().numpy()[np.zeros(n, dtype=int)], d, False, np.float32)
    for x, which in ((k, "k"), (v, "v")):
        for c, at in zip(caches, (slots, slots, alone)):
            codes, scales = O4.quantize(turned if which == "k" and c is caches[1] else x.float().cpu().numpy())
            assert (scales == O4.NAN_BYTE).sum() >= 6
            want = np.zeros(tuple(c.k[0].shape), dtype=np.uint8)
            for i, s in enumerate(at.tolist()):
                for h in range(H):
                    O4.store(want, which, s // B, h, s % B, codes[i, h], scales[i, h])
            assert np.array_equal(getattr(c, which)[0].cpu().numpy(), want), which
    for c in caches:
        assert c.device_error() == 0
        c.close()
