"""GPU: paged_query_attention and kv_append_rope_axes as they are used together, and calls at the edges of
how work is shared out: many sequences, rows named twice, row tiles that see nothing, two calls at once.

The oracle and the tolerance are test_gpu_query's: the attention is compared on the values the pool holds,
with queries read back from the rotation (whose own results test_gpu_rope_axes holds bit for bit)."""

import math

import numpy as np
import pytest
import torch

import test_gpu_query as G
from oracle import query as OQ
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_axes, rope_table

pytestmark = pytest.mark.gpu


def up(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).cuda()


class Served(G.Batch):
    """A cache whose tokens come from append_rope_axes: pages scattered, lengths grow."""

    def __init__(self, pool, d, H, B, room, seed=0):
        rng = self.rng = np.random.default_rng(seed)
        self.pool, self.d, self.H, self.B, self.lens = pool, d, H, B, [0] * len(room)
        per = [-(-c // B) for c in room]
        nb = sum(per) + 2
        ids = rng.permutation(nb).astype(np.int32)
        self.tab = np.full((len(room), max(per)), -1, dtype=np.int32)
        at = 0
        for s, m in enumerate(per):
            self.tab[s, :m] = ids[at:at + m]
            at += m
        self.cache = PagedKVCache(1, nb, B, H, d, pool)
        for t in self.cache.k + self.cache.v:
            t.view(torch.uint8).fill_(0x7F)                    # NaN where no token is
        self.ks = self.vs = None
        if pool == "fp8":
            for t in (self.cache.k_scale[0], self.cache.v_scale[0]):
                t.fill_(0.02)

    def slots(self, s, p):
        return self.tab[s][p // self.B].astype(np.int64) * self.B + p % self.B

    def read(self):
        k, v = self.cache.k[0], self.cache.v[0]
        bits = k.dtype not in (torch.float16, torch.float32)
        self.k, self.v = ((t.view(torch.uint8) if bits else t).cpu().numpy() for t in (k, v))
        if self.pool == "fp8":
            self.ks, self.vs = (t.cpu().numpy()[:self.cache.num_blocks] for t in (self.cache.k_scale[0], self.cache.v_scale[0]))


def expect(b, q, start, got, scale, cap=0.0, slopes=None, window=0):
    for s in range(len(start) - 1):
        rows = slice(start[s], start[s + 1])
        if start[s] == start[s + 1]:
            continue
        k, v = b.values(s, "k"), b.values(s, "v")
        want = OQ.query_attention(q[rows], k, v, scale, window, cap, slopes)
        t_max = (b.lens[s] * float(slopes.max()) if slopes is not None else 0.0) + (cap if cap else float(
            np.max(np.linalg.norm(q[rows], axis=-1))) * float(np.max(np.linalg.norm(k, axis=-1))) * scale)
        tol = G.tolerance(b.pool, q[rows].astype(np.float64), k, v, t_max, scale, cap, want)
        G.close(got[rows], want, tol, (s, start))


@pytest.mark.parametrize("pool", G.POOLS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_prompt_then_tokens(pool, cap):
    """A prompt whose positions have three axes, then single and drafted tokens, every step rotated, appended
    and attended, the later ones as one captured graph that reads its step's inputs."""
    d, H, Hq, B, axes = 128, 2, 8, 16, rope_axes([0] * 16 + [1] * 24 + [2] * 24)
    b = Served(pool, d, H, B, [400, 90, 30], seed=len(pool))
    table, scale = rope_table(512, d), 1 / math.sqrt(d)
    dt = np.float32 if pool == "f32" else np.float16
    ws, tab = b.cache.query_workspace(3, Hq, 4, 400), up(b.tab)          # (of single and drafted tokens)

    def step(new, run):
        start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        n = int(start[-1])
        q, k, v = (b.rng.standard_normal((n, h, d)).astype(dt) for h in (Hq, H, H))
        p = np.concatenate([np.arange(c, c + m) for c, m in zip(b.lens, new)])
        s = np.repeat(np.arange(len(new)), new)
        slots = np.array([b.slots(x, y) for x, y in zip(s, p)], dtype=np.int64)
        pos = np.stack((p, p // 7, p % 7))
        b.lens = [c + m for c, m in zip(b.lens, new)]
        q_out, out = run(new, torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                         up(slots, np.int64), up(pos), up(start), up(b.lens))
        torch.cuda.synchronize()
        assert b.cache.device_error() == 0
        b.read()
        expect(b, q_out.cpu().numpy(), start, out.cpu().numpy(), scale, cap)

    def eager(new, q, k, v, slots, pos, start, lens):
        q_out = b.cache.append_rope_axes(0, k, v, slots, pos, axes, table, q=q)
        kept = dict(workspace=ws, flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL) if max(new) <= 4 else {}
        return q_out, b.cache.query_attention(0, q_out, start, tab, lens, max(new), 400, scale, score_cap=cap, **kept)

    step([256, 70, 1], eager)                                  # prompts
    step([100, 0, 3], eager)                                   # a chunk with a prefix, nothing, a few
    for new in ([1, 1, 1], [4, 4, 4]):
        held = {}

        def captured(new, *now):
            if not held:
                held["in"] = [x.clone() for x in now]
                held["graph"] = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(held["graph"]):
                    held["out"] = eager(new, *held["in"])
            for x, y in zip(held["in"], now):
                x.copy_(y)
            held["graph"].replay()
            return held["out"]

        for _ in range(3):
            step(new, captured)
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
def test_many_sequences(pool):
    """More sequences than one launch of the few-row kernel takes, some of them empty."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(2, 40, 2100)]
    b = G.Batch(pool, 64, 1, 8, lens, seed=2)
    new = [int(x) for x in rng.integers(0, 3, 2100)]
    G.run(b, new, 2, gap=5)
    G.run(b, [1] * 2100, 1, slopes=True)
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "int4"])
@pytest.mark.parametrize("slopes", [False, True])
def test_row_tiles_that_see_nothing(pool, slopes):
    """Of a pair of row tiles the first, the second or both; several such pairs one after the other."""
    new, lens = [1400, 300], [1500, 300]
    b = G.Batch(pool, 64, 1, 16, lens, seed=3)
    p = np.concatenate([np.arange(c - n, c) for n, c in zip(new, lens)])
    r = np.stack((np.zeros_like(p), p + 1), 1)
    row = np.arange(len(p))
    r[(row >= 128) & (row < 384)] = (7, 7)                     # the first pair's second tile, the second's first
    r[(row >= 512) & (row < 1280)] = (0, -3)                   # three pairs
    r[1400 + 255:] = (300, 200)                                # the last ones
    G.run(b, new, 1, ranges=r, slopes=slopes)
    r[:] = (5, 5)
    got, _, _ = G.run(b, new, 1, ranges=r, slopes=slopes, check=False)
    assert not got.any()
    b.cache.close()


def test_rows_named_twice():
    """query_start that goes back: the sequences that begin after their end are left out and reported; the
    others, more of them together than there are rows, are all done."""
    b = G.Batch("f16", 128, 2, 16, [300] * 9, seed=4)
    b.tab[:] = b.tab[0]
    rng = np.random.default_rng(1)
    q = rng.standard_normal((300, 4, 128)).astype(np.float16)
    for n in (300, 4):
        out = torch.full((300, 4, 128), 7.5, dtype=torch.float16, device="cuda")
        b.cache.query_attention(0, torch.from_numpy(q).cuda(), up([0, n] * 5), up(b.tab), up([300] * 9), n, 300, 0.09, out=out)
        assert b.cache.device_error() == abi.KV_DEVERR_QUERY
        got = out.cpu().numpy()
        k, v = b.values(0, "k"), b.values(0, "v")
        want = OQ.query_attention(q[:n], k, v, 0.09)
        G.close(got[:n], want, G.tolerance("f16", q[:n].astype(np.float64), k, v, 40.0, 0.09, 0.0, want), n)
        assert (got[n:] == 7.5).all()
    b.cache.close()


@pytest.mark.parametrize("pool", ["f32", "f16", "fp8", "int4"])
def test_steep_and_rising_slopes(pool):
    """Distance terms of hundreds per step, of either sign: the nearest, or the farthest, position takes all."""
    b = G.Batch(pool, 128, 2, 16, [700, 260, 33], seed=6)
    sl = np.array([300.0, 8.0, -0.5, -40.0], dtype=np.float32)
    for new in ([500, 260, 33], [1, 2, 3]):
        q = b.rng.standard_normal((sum(new), 4, 128)).astype(np.float32 if pool == "f32" else np.float16)
        start = np.concatenate(([0], np.cumsum(new)))
        out = b.cache.query_attention(0, torch.from_numpy(q).cuda(), up(start), up(b.tab), up(b.lens), max(new), 700, 0.09,
                                      slopes=up(sl, np.float32))
        assert b.cache.device_error() == 0
        got = out.cpu().numpy()
        for s, m in enumerate(new):
            rows = slice(start[s], start[s + 1])
            k, v = b.values(s, "k"), b.values(s, "v")
            want = OQ.query_attention(q[rows], k, v, 0.09, 0, 0.0, sl)
            # the scores that count lie within 200 of the largest, and that one is rounded at its own size
            t_max = 40.0 * b.lens[s] + 40.0
            tol = G.tolerance(pool, q[rows].astype(np.float64), k, v, t_max, 0.09, 0.0, want)
            G.close(got[rows], want, tol, (s, m))
    b.cache.close()


@pytest.mark.parametrize("new", [[260, 130], [2, 1]])
def test_two_calls_at_once(new):
    """Two streams with a workspace each: the bits of a call by itself."""
    b = G.Batch("fp8", 128, 2, 16, [3000, 900], seed=7)
    want, q, _ = G.run(b, new, 4)
    tq, st, tab, ln = torch.from_numpy(q).cuda(), up(np.concatenate(([0], np.cumsum(new)))), up(b.tab), up(b.lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [b.cache.query_workspace(2, 8, max(new), 3000) for _ in streams]
    outs = [torch.zeros_like(tq) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, o in zip(streams, ws, outs):
            b.cache.query_attention(0, tq, st, tab, ln, max(new), 3000, 1 / math.sqrt(128), out=o, workspace=w, stream=s,
                                    flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL)
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(o.cpu().numpy(), want)
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
@pytest.mark.parametrize("d,group", [(128, 8), (64, 1)])
def test_contexts_cut_into_parts(pool, d, group):
    """Few rows over long contexts: parts of the keys, joined.  Masks that leave parts, rows and row tiles empty, a
    window within one part, a short sequence beside a long one, a workspace kept and one that is given zeroed."""
    new, lens = [40, 300, 20, 1], [3000, 1700, 21, 900]
    b = G.Batch(pool, d, 1, 16, lens, seed=d + group)
    want, q, _ = G.run(b, new, group)
    ws = b.cache.query_workspace(4, group, 300, 3000, num_tokens=sum(new))
    assert ws.numel() > sum(new) * group * d * 8
    got, _, _ = G.run(b, new, group, workspace=ws, flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL, check=False, q_in=q)
    assert np.array_equal(got, want)
    G.run(b, new, group, cap=20.0, qmul=3.0, gap=4)
    G.run(b, new, group, slopes=True)
    G.run(b, new, group, window=100)
    p = np.concatenate([np.arange(c - n, c) for n, c in zip(new, lens)])
    r = np.stack((p // 700 * 700, p + 1), 1)
    r[3::5] = (600, 610)
    r[4::5] = (9, 9)
    r[40:168] = (0, 0)                                         # a whole row tile with one head, most of one with eight
    G.run(b, new, group, ranges=r)
    G.run(b, new, group, ranges=r, slopes=True)
    # what one row may not see: NaN within a part that others of its tile see
    blk = b.tab[0][2990 // 16]
    if pool == "f16":
        b.k[blk, :, 2990 % 16], b.v[blk, :, 2990 % 16] = np.nan, np.nan
        b.upload()
        got, q, _ = G.run(b, new, group, check=False)
        k, v = b.values(0, "k")[:2990], b.values(0, "v")[:2990]
        assert np.isnan(got[30:40]).all()
        want = OQ.query_attention(q[:30], k, v, 1 / math.sqrt(d))
        tol = G.tolerance(pool, q[:30].astype(np.float64), k, v, 40.0, 1 / math.sqrt(d), 0.0, want)
        G.close(got[:30], want, tol, "beside NaN")
    b.cache.close()
