"""GPU: decode attention over 4-bit pools asks for workspace by what its CTAs may leave unfinished."""

import numpy as np
import pytest
import torch

import test_gpu_int4 as T
from paged_kv_cache_169_gb300 import abi

pytestmark = pytest.mark.gpu


def test_many_short_sequences_fit_the_static_scratch():
    """1024 sequences of 40 heads whose contexts no CTA shares with another: the static entry takes
    them, and gives the bits of the call with a workspace."""
    rng = np.random.default_rng(1)
    lens, H, d, B = [int(n) for n in rng.integers(1, 25, 1024)], 40, 128, 8
    cache, tab, pools = T.build(rng, lens, H, d, B)
    T.to_cache(cache, pools)
    q = torch.from_numpy(rng.standard_normal((1024, H, d)).astype(np.float16)).cuda()
    tabs, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = cache.attention(0, q, tabs, ln, 24, 0.1)
    out = torch.zeros_like(want)
    abi.paged_decode_attention_static(cache.handle, 0, q.data_ptr(), out.data_ptr(), tabs.data_ptr(), tabs.shape[1],
                                      ln.data_ptr(), 1024, 24, 0.1, 0, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, want) and cache.device_error() == 0
    pick = [0, 511, 1023]
    w, tol = T.oracle(pools, tab[pick], [lens[s] for s in pick], q[pick].cpu().numpy(), B, d, 0.1)
    assert np.max(np.abs(out[pick].double().cpu().numpy() - w)) <= tol
    cache.close()


@pytest.mark.parametrize("G,d", [(1, 128), (8, 64)])
def test_workspace_does_not_grow_with_the_batch(G, d):
    cache, _, _ = T.build(np.random.default_rng(2), [1], 4, d, 8)
    size = [abi.paged_decode_workspace_size_gqa(cache.handle, s, 4 * G, 4096, 0) for s in (1, 64, 1024, 5000)]
    assert 0 < size[0] and max(size) <= 4 << 20
    cache.close()


@pytest.mark.parametrize("G,d,B", [(1, 128, 16), (2, 64, 8), (8, 128, 32)])
def test_units_that_cross_ctas_side_by_side(G, d, B):
    """Contexts of about a CTA's share each, so that nearly every CTA ends one unit and begins another,
    with long ones that take many CTAs between them; a kept zeroed workspace, twice: the same bits."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(300, 900, 90)]
    lens[7], lens[40], lens[41], lens[89] = 20_000, 9_000, 0, 5_000
    cache, tab, pools = T.build(rng, lens, 2, d, B)
    T.to_cache(cache, pools)
    q = rng.standard_normal((len(lens), 2 * G, d)).astype(np.float16)
    t = [torch.from_numpy(x).cuda() for x in (q, tab, np.array(lens, dtype=np.int32))]
    ws = cache.zeroed_workspace(len(lens), 20_000, num_q_heads=2 * G)
    outs = [cache.attention_ex(0, *t, 20_000, 0.1, workspace=ws, flags=abi.KV_DECODE_WORKSPACE_ZEROED).clone()
            for _ in range(2)]
    assert torch.equal(outs[0], outs[1]) and cache.device_error() == 0
    pick = [6, 7, 8, 39, 40, 41, 42, 88, 89]
    want, tol = T.oracle(pools, tab[pick], [lens[s] for s in pick], q[pick], B, d, 0.1)
    assert np.max(np.abs(outs[0][pick].double().cpu().numpy() - want)) <= tol
    cache.close()
