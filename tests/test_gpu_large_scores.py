"""GPU: scores so large that float32 neighbours are 16 apart, float16 and FP8 pools."""

import numpy as np
import pytest
import torch

from paged_kv_cache_169_gb300.cache import PagedKVCache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,B", [(128, 16), (64, 8)])
@pytest.mark.parametrize("H", [1, 2, 4])
def test_float16_pools(d, B, H):
    """Two tokens, chunks apart, with scores of 16384 k0 and 8 k1 more (both exact in float32), for many
    k0 and k1; every other token's score is far below.  The later token's weight is at least 2980 times
    the other's; in float32 its score lies 0, 16 or 32 above in log2 units, each rounding half a step (8),
    so its share of the weights is anything between a half and all."""
    n = 100
    cache = PagedKVCache(1, -(-n // B), B, H, d, "f16")
    tab = torch.arange(-(-n // B), dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    slots = torch.arange(n, device="cuda")
    q = torch.zeros(1, H, d, device="cuda").half()
    q[..., 0], q[..., 7] = 16384, 8
    v = torch.randn(n, H, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    for k0 in range(5700, 8192, 60):
        for k1 in (1, 2, 3):
            k = torch.zeros(n, H, d, device="cuda").half()
            k[..., 0] = -8000
            k[3, :, 0] = k[90, :, 0] = k0
            k[90, :, 7] = k1
            cache.append(0, k, v, slots)
            out = cache.attention(0, q, tab, lens, n, 1.0).cpu()
            a, b = v[3].float().cpu(), v[90].float().cpu()
            far = torch.maximum((out[0] - b).abs(), (out[0] - (a + b) / 2).abs())
            assert torch.all(far <= (a - b).abs() / 2 + 1e-3 * (a.abs() + b.abs())), (k0, k1)
    assert cache.device_error() == 0
    cache.close()
