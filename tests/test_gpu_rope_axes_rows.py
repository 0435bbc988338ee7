"""GPU: append_rope_axes with rows of positions that no pair uses, and with an abi.kv_rope_axes made by hand: the same bits as
with the rows in use and rope_axes."""

import pytest
import torch

from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_axes, rope_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs,used", [([0] * 32, 1), ([0, 1] * 16, 2), ([1] * 32, 2)])
def test_rows_that_no_pair_uses(pairs, used):
    n = 21
    cache = PagedKVCache(1, 4, 8, 2, 64, "f16")
    torch.manual_seed(0)
    k, v, q = (torch.randn(n, 2, 64, device="cuda").half() for _ in range(3))
    slots, tab = torch.randperm(32, device="cuda")[:n], rope_table(50, 64)
    pos = torch.randint(0, 50, (3, n), dtype=torch.int32, device="cuda")
    pos[used:] = -7                                            # (not looked at)
    by_hand = abi.kv_rope_axes(used, 0)
    by_hand.pair_axis[:32] = pairs
    res = []
    for p, axes in ((pos[:used].contiguous(), rope_axes(pairs)), (pos, rope_axes(pairs)), (pos, by_hand)):
        for t in (cache.k[0], cache.v[0]):
            t.zero_()
        out = cache.append_rope_axes(0, k, v, slots, p, axes, tab, q=q)
        assert cache.device_error() == 0
        res.append([out.clone(), cache.k[0].clone(), cache.v[0].clone()])
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, res[0]))
    for bad in (pos[:used - 1], pos[:, :n - 1].contiguous(), pos[0]):
        with pytest.raises(ValueError):
            cache.append_rope_axes(0, k, v, slots, bad, rope_axes(pairs), tab)
    cache.close()
