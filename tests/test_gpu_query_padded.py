"""GPU: paged_query_attention on a padded buffer of queries (more rows than the sequences use) after long contexts, whose
keys are cut into parts: right, and nothing behind the workspace is written.  Oracle and tolerance: test_gpu_query's."""

import math

import numpy as np
import pytest
import torch

import test_gpu_query as G
from oracle import query as OQ
from paged_kv_cache_169_gb300 import abi

pytestmark = pytest.mark.gpu


def up(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).cuda()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
@pytest.mark.parametrize("d,H,group,lens,new,tokens", [
    (128, 4, 4, [5000], [83], 2048),                           # one sequence in a buffer of 2048 rows
    (128, 2, 8, [3000, 1500], [100, 37], 1024),
    (64, 2, 1, [4000, 2000, 900], [17, 40, 0], 400),
    (64, 1, 2, [2600], [300], 301),                            # one row more than is used
])
def test_few_rows_of_a_padded_buffer(pool, d, H, group, lens, new, tokens):
    b = G.Batch(pool, d, H, 16, lens, seed=d + group)
    Hq, most, scale = H * group, max(new), 1 / math.sqrt(d)
    q = b.rng.standard_normal((tokens, Hq, d)).astype(np.float16)
    start = np.concatenate(([0], np.cumsum(new))) + 1 if tokens - sum(new) > 1 else np.concatenate(([0], np.cumsum(new)))
    a = abi.kv_query_args()
    a.num_q_heads, a.batch, a.max_queries, a.max_context, a.num_tokens = Hq, len(lens), most, max(lens), tokens
    need = abi.paged_query_workspace_size(b.cache.handle, a)
    room = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    tq, st, tab, ln = torch.from_numpy(q).cuda(), up(start), up(b.tab), up(b.lens)
    for ws in (room[:need], None):
        out = torch.full((tokens, Hq, d), 7.5, dtype=torch.float16, device="cuda")
        b.cache.query_attention(0, tq, st, tab, ln, most, max(lens), scale, out=out, workspace=ws)
        assert b.cache.device_error() == 0
        assert (room[need:] == 0xA5).all()
        got = out.cpu().numpy()
        assert (got[:start[0]] == 7.5).all() and (got[start[-1]:] == 7.5).all()
        for s, m in enumerate(new):
            rows = slice(start[s], start[s + 1])
            if m == 0:
                continue
            k, v = b.values(s, "k"), b.values(s, "v")
            want = OQ.query_attention(q[rows], k, v, scale)
            t_max = float(np.max(np.linalg.norm(q[rows].astype(np.float64), axis=-1)) * np.max(np.linalg.norm(k, axis=-1))) * scale
            G.close(got[rows], want, G.tolerance(pool, q[rows].astype(np.float64), k, v, t_max, scale, 0.0, want), (s, m))
    b.cache.close()


def test_rows_named_twice_in_parts():
    """Sequences that share rows of q, their keys cut into parts: those that end before they begin are left out, the
    others' rows are all done (their results are the same ones here)."""
    b = G.Batch("f16", 128, 2, 16, [3000] * 3, seed=4)
    b.tab[:] = b.tab[0]
    n, scale = 40, 1 / math.sqrt(128)
    q = b.rng.standard_normal((500, 4, 128)).astype(np.float16)
    out = torch.full((500, 4, 128), 7.5, dtype=torch.float16, device="cuda")
    b.cache.query_attention(0, torch.from_numpy(q).cuda(), up([0, n, 0, n]), up(b.tab), up([3000] * 3), n, 3000, scale, out=out)
    assert b.cache.device_error() == abi.KV_DEVERR_QUERY
    got = out.cpu().numpy()
    k, v = b.values(0, "k"), b.values(0, "v")
    want = OQ.query_attention(q[:n], k, v, scale)
    G.close(got[:n], want, G.tolerance("f16", q[:n].astype(np.float64), k, v, 40.0, scale, 0.0, want), n)
    assert (got[n:] == 7.5).all()
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
@pytest.mark.parametrize("lens", [[700, 90], [3000, 400]])
def test_one_workspace_for_prompts_and_tokens(pool, lens):
    """The workspace of the largest prompt, zeroed once, serves prompts and the single tokens between them."""
    b = G.Batch(pool, 128, 2, 16, lens, seed=len(pool))
    ws = b.cache.query_workspace(2, 4, 90, max(lens))
    flags = abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL
    for new in ([90, 60], [1, 1], [20, 3], [1, 2], [90, 60]):
        want, q, _ = G.run(b, new, 2)
        for _ in range(2):
            assert np.array_equal(G.run(b, new, 2, workspace=ws, flags=flags, check=False, q_in=q)[0], want)
    b.cache.close()
