"""GPU: paged_query_attention with windows up to the largest int, which see everything, also from positions before 0 (fewer
cached tokens than rows, with ranges of their own).  Oracle and tolerance: test_gpu_query's."""

import numpy as np
import pytest
import torch

import test_gpu_query as G
from oracle import query as OQ
from paged_kv_cache_169_gb300 import abi

pytestmark = pytest.mark.gpu


def up(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


@pytest.mark.parametrize("pool", G.POOLS)
@pytest.mark.parametrize("new", [40, 4])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 20, 2 ** 25, 2 ** 24, 100])
def test_large_windows_from_before_the_context(pool, new, window):
    c = new - 3                                                # the first three rows stand at -3, -2 and -1
    b = G.Batch(pool, 64, 2, 8, [c], seed=new)
    q = b.rng.standard_normal((new, 4, 64)).astype(np.float32 if pool == "f32" else np.float16)
    ranges = np.tile(np.array([[0, c]], dtype=np.int32), (new, 1))
    got = b.cache.query_attention(0, torch.from_numpy(q).cuda(), up([0, new]), up(b.tab), up([c]), new, c, 0.125, window=window,
                                  ranges=up(ranges)).cpu().numpy()
    assert b.cache.device_error() == abi.KV_DEVERR_CONTEXT
    k, v = b.values(0, "k"), b.values(0, "v")
    want = OQ.query_attention(q, k, v, 0.125, window, ranges=ranges)
    G.close(got, want, G.tolerance(pool, q.astype(np.float64), k, v, 40.0, 0.125, 0.0, want), window)
    b.cache.close()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 24 + 1])
def test_large_windows(window):
    b = G.Batch("f16", 128, 1, 16, [300, 50], seed=1)
    for new in ([200, 50], [1, 2]):
        G.run(b, new, 2, window=window)
    b.cache.close()
