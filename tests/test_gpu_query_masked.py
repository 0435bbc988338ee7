"""GPU: paged_query_attention where what some rows do not see is not finite, in units of work that several CTAs share: a row
that came out not finite is worked out again, by the CTA that joins the unit's parts, often two units one after the other.
Oracle and tolerance: test_gpu_query's."""

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
@pytest.mark.parametrize("seqs,H,c", [(37, 4, 700), (19, 8, 1200), (50, 2, 500), (3, 1, 6000)])
def test_units_of_several_ctas(pool, seqs, H, c):
    """Two rows a sequence; the last token's key and value are NaN, which the last row alone sees: it is NaN, the one
    before it is right, in every unit and every time."""
    d, B, scale = 64, 16, 0.125
    lens = [c + 16 * (s % 7) + s for s in range(seqs)]
    b = G.Batch(pool, d, H, B, lens, seed=seqs)
    blk, off = np.array([b.tab[s][(n - 1) // B] for s, n in enumerate(lens)]), np.array([(n - 1) % B for n in lens])
    for i, o in zip(blk, off):
        if pool == "int4":
            t = o % 8
            b.k[i, :, o // 8, 4 * d + t * 4:4 * d + t * 4 + 4] = G.O4.NAN_BYTE
            b.v[i, :, o // 8, 4 * d + t::8] = G.O4.NAN_BYTE
        else:
            bad = 0x7F if pool == "fp8" else np.nan
            b.k[i, :, o], b.v[i, :, o] = bad, bad
    b.upload()
    q = b.rng.standard_normal((2 * seqs, H, d)).astype(np.float16)
    want, tol = [], []
    for s, n in enumerate(lens):
        k, v = b.values(s, "k")[:n - 1], b.values(s, "v")[:n - 1]
        want.append(OQ.query_attention(q[2 * s:2 * s + 1], k, v, scale))
        t_max = float(np.max(np.linalg.norm(q[2 * s].astype(np.float64), axis=-1)) * np.max(np.linalg.norm(k, axis=-1))) * scale
        tol.append(G.tolerance(pool, q[2 * s:2 * s + 1].astype(np.float64), k, v, t_max, scale, 0.0, want[-1]))
    want, tol = np.concatenate(want), np.concatenate(tol)
    tq, st, tab, ln = torch.from_numpy(q).cuda(), up(np.arange(0, 2 * seqs + 1, 2)), up(b.tab), up(lens)
    ws = b.cache.query_workspace(seqs, H, 2, max(lens))
    outs = [torch.zeros_like(tq) for _ in range(30)]
    for out in outs:
        b.cache.query_attention(0, tq, st, tab, ln, 2, max(lens), scale, out=out, workspace=ws,
                                flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL)
    assert b.cache.device_error() == 0
    for out in outs:
        got = out.cpu().numpy()
        assert np.isnan(got[1::2]).all()
        G.close(got[0::2], want, tol, pool)
        assert np.array_equal(got[0::2], outs[0].cpu().numpy()[0::2])
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
@pytest.mark.parametrize("d,group", [(128, 8), (64, 1)])
def test_rows_of_joined_parts(pool, d, group):
    """Keys cut into parts: NaN at positions that only the last rows see, in the last part and before it.  Every row that
    does not see them is right where the join works it out again, the same bits every time."""
    n, c, B, scale = 60, 3000, 16, 1 / math.sqrt(d)
    b = G.Batch(pool, d, 1, B, [c], seed=d)
    for p in (c - 1, c - 20):
        i, o = b.tab[0][p // B], p % B
        if pool == "int4":
            b.k[i, :, o // 8, 4 * d + o % 8 * (d // 16):4 * d + (o % 8 + 1) * (d // 16)] = G.O4.NAN_BYTE
            b.v[i, :, o // 8, 4 * d + o % 8::8] = G.O4.NAN_BYTE
        else:
            bad = 0x7F if pool == "fp8" else np.nan
            b.k[i, :, o], b.v[i, :, o] = bad, bad
    b.upload()
    q = b.rng.standard_normal((n, group, d)).astype(np.float16)
    k, v = b.values(0, "k"), b.values(0, "v")
    m = n - 20                                                 # rows that see neither
    args = (up([0, n]), up(b.tab), up([c]), n, c, scale)
    first = None
    for _ in range(10):
        got = b.cache.query_attention(0, torch.from_numpy(q).cuda(), *args).cpu().numpy()
        assert b.cache.device_error() == 0
        assert np.isnan(got[m:]).all()
        first = got if first is None else first
        assert np.array_equal(got[:m], first[:m])
    kk, vv = k[:c - 20], v[:c - 20]
    want = np.concatenate([OQ.query_attention(q[i:i + 1], kk[:c - n + i + 1], vv[:c - n + i + 1], scale) for i in range(m)])
    t_max = float(np.max(np.linalg.norm(q.astype(np.float64), axis=-1)) * np.max(np.linalg.norm(kk, axis=-1))) * scale
    G.close(first[:m], want, G.tolerance(pool, q.astype(np.float64), kk, vv, t_max, scale, 0.0, want), pool)
    b.cache.close()


def test_rows_worked_out_again_over_a_long_context():
    """The last token's key and value are NaN after 250 000 others: the rows of its row tiles that do not see it are worked
    out again, 16 a warp, for longer than a wait lasts that nothing moves beside.  No wait runs out, and the rows are right."""
    c, n, H, group, d, B, scale = 250_000, 512, 8, 8, 64, 32, 0.125
    nb = -(-c // B)
    cache = G.PagedKVCache(1, nb, B, H, d, "fp8")
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in (cache.k[0], cache.v[0]):
        t.view(torch.uint8).copy_(torch.randint(0, 127, t.shape, dtype=torch.uint8, device="cuda", generator=gen))
        t.view(torch.uint8).bitwise_or_(torch.randint(0, 2, t.shape, dtype=torch.uint8, device="cuda", generator=gen) << 7)
        t.view(torch.uint8)[(c - 1) // B, :, (c - 1) % B] = 0x7F
    cache.k_scale[0].fill_(0.004)
    cache.v_scale[0].fill_(0.01)
    q = rng.standard_normal((n, H * group, d)).astype(np.float16)
    got = cache.query_attention(0, torch.from_numpy(q).cuda(), up([0, n]), up(np.arange(nb)[None]), up([c]), n, c,
                                scale).cpu().numpy()
    assert cache.device_error() == 0
    assert np.isnan(got[-1]).all() and not np.isnan(got[:-1]).any()
    for head in (0, 29, 63):
        k, v = (G.OF.decode(t.view(torch.uint8)[:, head // group].reshape(-1, d)[:c - 1].cpu().numpy()) * s
                for t, s in ((cache.k[0], float(cache.k_scale[0][0])), (cache.v[0], float(cache.v_scale[0][0]))))
        for i in (0, n - 3, n - 2):
            seen = c - n + i + 1
            want = OQ.query_attention(q[i:i + 1, head:head + 1], k[:seen, None], v[:seen, None], scale)     # (its last row)
            tol = G.tolerance("fp8", q[i:i + 1, head:head + 1].astype(np.float64), k[:seen, None], v[:seen, None], 60.0, scale, 0.0,
                              want)
            G.close(got[i:i + 1, head:head + 1], want, tol, (head, i))
    cache.close()
