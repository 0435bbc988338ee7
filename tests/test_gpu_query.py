"""GPU: paged_query_attention against the float64 oracle on the values the pool holds.

Tolerance, derived.  With weights w_t and values v_t a row is sum w v / sum w.  The weights enter the
sums of values as float16: off by half a step, 2^-11 relative, which moves the row by at most 2^-11
max|v|; a relative error e of every weight (in both sums) by at most 2 e max|v|.  e: the score's
roundings.  A float32 sum of d products in any order, each addition off by 2^-23 of sum |q||k| at most
(the tensor core may truncate), times scale; a cap evaluates tanh within 2^-20 of the cap; the
multiplications and the distance term round t (2^-22 of |t|); the exponential is good to 2^-22.  Weights
below the normal float16 ones are off by 2^-25 where the largest is 2^7 or more: n 2^-32 in all.  Sums over
n keys: one rounding per 16 of them and per joined part, (n/16 + 64) 2^-23.  The result is rounded once:
2^-11 of it (float32 pools: no float16 anywhere, 2^-24)."""

import math

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import int4 as O4
from oracle import query as OQ
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache

pytestmark = pytest.mark.gpu

POOLS = ["f32", "f16", "fp8", "int4"]


class Batch:
    """A cache holding the given contexts, poisoned (NaN) wherever no sequence holds a token."""

    def __init__(self, pool, d, H, B, lens, seed=0, spare=2, vscale=(0.004, 0.02)):
        rng = self.rng = np.random.default_rng(seed)
        self.pool, self.d, self.H, self.B, self.lens = pool, d, H, B, list(lens)
        per = [-(-c // B) for c in self.lens]
        nb = sum(per) + spare
        perm = rng.permutation(nb).astype(np.int32)
        self.tab = np.full((len(self.lens), max(per + [1]) + 1), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(per):
            self.tab[s, :k] = perm[at:at + k]
            at += k
        self.cache = PagedKVCache(1, nb, B, H, d, pool)
        shape = tuple(self.cache.k[0].shape)
        used = np.zeros((nb, B), dtype=bool)
        for s, c in enumerate(self.lens):
            p = np.arange(c)
            used[self.tab[s][p // B], p % B] = True
        self.k, self.v = (self._fill(shape, used, w) for w in "kv")
        self.ks = self.vs = None
        if pool == "fp8":
            self.ks = rng.uniform(0.004, 0.02, nb).astype(np.float32)
            self.vs = rng.uniform(*vscale, nb).astype(np.float32)
        self.upload()

    def _fill(self, shape, used, which):
        rng, d = self.rng, self.d
        if self.pool == "int4":
            a = rng.integers(0, 256, shape, dtype=np.uint8)
            a[..., 4 * d:] = rng.integers(85, 107, a[..., 4 * d:].shape)
            for b, o in zip(*np.nonzero(~used)):
                t = o % 8
                if which == "k":
                    a[b, :, o // 8, 4 * d + t * (d // 16):4 * d + (t + 1) * (d // 16)] = O4.NAN_BYTE
                else:
                    a[b, :, o // 8, 4 * d + t::8] = O4.NAN_BYTE
            return a
        x = rng.standard_normal(shape).astype(np.float32)
        if self.pool == "fp8":
            a = OF.encode(np.clip(x * 110, -448, 448)).astype(np.uint8)
            a[np.broadcast_to(~used[:, None, :, None], shape)] = 0x7F
            return a
        a = x.astype(np.float16 if self.pool == "f16" else np.float32)
        a[np.broadcast_to(~used[:, None, :, None], shape)] = np.nan
        return a

    def upload(self):
        self.cache.k[0].copy_(torch.from_numpy(self.k))
        self.cache.v[0].copy_(torch.from_numpy(self.v))
        if self.ks is not None:
            nb = len(self.ks)
            self.cache.k_scale[0][:nb].copy_(torch.from_numpy(self.ks))
            self.cache.v_scale[0][:nb].copy_(torch.from_numpy(self.vs))

    def values(self, s, which):
        """float64 [c, H, d] of sequence s."""
        a, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        p = np.arange(self.lens[s])
        blk, off = self.tab[s][p // self.B], p % self.B
        if self.pool == "int4":
            return O4.token_values(a, which, self.d, blk, off)
        x = a[blk, :, off]
        if self.pool == "fp8":
            return OF.decode(x) * sc[blk].astype(np.float64)[:, None, None]
        return x.astype(np.float64)


def tolerance(pool, q, k, v, t_max, scale, cap, want):
    d, n = q.shape[-1], max(1, k.shape[0])
    mag = float(np.max(np.abs(q).sum(-1))) * float(np.max(np.abs(k))) * scale
    mag = min(mag, float(np.max(np.linalg.norm(q, axis=-1))) * float(np.max(np.linalg.norm(k, axis=-1))) * scale)
    e = (d + 8) * 2.0 ** -23 * mag + cap * 2.0 ** -20 + t_max * 2.0 ** -22 + 2.0 ** -22 + (n / 16 + 64) * 2.0 ** -23
    half = 2.0 ** -24 if pool == "f32" else 2.0 ** -11
    return 2 * e * float(np.max(np.abs(v))) + (0.0 if pool == "f32" else (half + n * 2.0 ** -32) * float(np.max(np.abs(v)))) \
        + half * np.abs(want) + 2.0 ** -25


def close(got, want, tol, what):
    """Every element within its tolerance.  A result that rounds beyond float16's largest value, 65504, is
    infinite: 448 * 200 is a value that an FP8 pool holds."""
    got, beyond = got.astype(np.float64), np.abs(want) + tol >= 65504
    assert (~beyond | (got * np.sign(want) >= np.minimum(np.abs(want) - tol, 65504))).all(), what
    worst = float(np.max(np.where(beyond, 0.0, np.abs(got - want)) / tol))
    assert worst <= 1, (what, worst)


def run(b, new, G, window=0, cap=0.0, slopes=False, ranges=None, scale=None, qmul=1.0, packed=False, gap=0, stream=None,
        workspace=None, flags=0, check=True, q_in=None):
    """Call and compare every row; rows of no sequence (gap rows after the last one) must stay as they were."""
    rng, d, H = b.rng, b.d, b.H
    Hq, n = H * G, int(sum(new)) + gap
    dt = np.float32 if b.pool == "f32" else np.float16
    q = (rng.standard_normal((n, Hq, d)) * qmul).astype(dt) if q_in is None else q_in
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    tq = torch.from_numpy(q).cuda()
    if packed:
        wide = torch.full((n, Hq + 2, d), float("nan"), dtype=tq.dtype, device="cuda")
        wide[:, :Hq] = tq
        tq = wide[:, :Hq]
    out = torch.full((n, Hq + (3 if packed else 0), d), 7.5, dtype=tq.dtype, device="cuda")
    start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    sl = rng.uniform(0.01, 0.6, Hq).astype(np.float32) if slopes else None
    up = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()       # noqa: E731
    args = (up(start), up(b.tab), up(np.array(b.lens, dtype=np.int32)), max(list(new) + [0]), max(b.lens + [0]), scale)
    more = dict(slopes=up(sl), ranges=up(None if ranges is None else ranges.astype(np.int32)))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    b.cache.query_attention(0, tq, *args, window=window, score_cap=cap, out=out[:, :Hq], workspace=workspace, flags=flags,
                            stream=stream, **more)
    if stream is not None:
        stream.synchronize()
    assert b.cache.device_error() == 0
    got = out.cpu().numpy()
    assert (got[start[-1]:] == 7.5).all() and (got[:, Hq:] == 7.5).all()
    if not check:
        return got[:, :Hq], q, sl
    for s, m in enumerate(new):
        rows = slice(start[s], start[s + 1])
        if m == 0:
            continue
        k, v = b.values(s, "k"), b.values(s, "v")
        want = OQ.query_attention(q[rows], k, v, scale, window, cap, sl, None if ranges is None else ranges[rows])
        if not len(k):
            assert not got[rows, :Hq].any()
            continue
        far = b.lens[s] * float(sl.max()) if slopes else 0.0
        t_max = far + (cap if cap else float(np.max(np.linalg.norm(q[rows], axis=-1))) *
                       float(np.max(np.linalg.norm(k, axis=-1))) * scale)
        tol = tolerance(b.pool, q[rows].astype(np.float64), k, v, min(t_max, far + 200.0), scale, cap, want)
        close(got[rows, :Hq], want, tol, (s, m, b.lens[s]))
    return got[:, :Hq], q, sl


MIXED_NEW = [1, 5, 0, 17, 130, 3, 64, 1, 257, 2]
MIXED_LEN = [1, 5, 20, 40, 130, 300, 193, 257, 500, 129]


def prefix_ranges(new, lens):
    out = []
    for n, c in zip(new, lens):
        p = np.arange(c - n, c)
        out.append(np.stack((np.zeros_like(p), np.maximum(p + 1, c - n + n // 2)), 1))
    return np.concatenate(out)


def doc_ranges(new, lens, size=50):
    out = []
    for n, c in zip(new, lens):
        p = np.arange(c - n, c)
        out.append(np.stack((p // size * size, p + 1), 1))
    return np.concatenate(out)


def wild_ranges(new, lens, rng):
    """Any intervals: empty, reversed, beyond the context, before it."""
    n = int(sum(new))
    r = np.stack((rng.integers(-50, 200, n), rng.integers(-50, 400, n)), 1)
    r[::7] = (2 ** 31 - 1, -2 ** 31)
    r[3::11] = (-2 ** 31, 2 ** 31 - 1)
    return r


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("d,B,H,G", [(128, 16, 3, 1), (64, 8, 2, 4), (128, 8, 1, 8), (64, 32, 2, 2), (128, 32, 2, 2),
                                     (64, 16, 3, 1)])
def test_mixed_lengths(pool, d, B, H, G):
    b = Batch(pool, d, H, B, MIXED_LEN, seed=d + B + G)
    run(b, MIXED_NEW, G, packed=G == 4, gap=3)
    b.cache.close()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("cap,slopes,window", [(50.0, False, 0), (3.0, True, 0), (0.0, True, 70), (0.0, False, 33),
                                               (30.0, True, 129)])
def test_score_forms(pool, cap, slopes, window):
    b = Batch(pool, 128, 2, 16, MIXED_LEN, seed=int(cap) + window)
    run(b, MIXED_NEW, 2, window=window, cap=cap, slopes=slopes, qmul=4.0 if cap else 1.0)
    b.cache.close()
    b = Batch(pool, 64, 2, 8, [40, 16, 300], seed=3)
    run(b, [1, 16, 4], 1, window=window, cap=cap, slopes=slopes, qmul=4.0 if cap else 1.0)
    b.cache.close()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("kind", ["prefix", "docs", "wild"])
@pytest.mark.parametrize("slopes,window", [(False, 0), (True, 0), (False, 40)])
def test_ranges(pool, kind, slopes, window):
    b = Batch(pool, 128, 2, 16, MIXED_LEN, seed=11)
    r = {"prefix": prefix_ranges, "docs": doc_ranges}.get(kind)
    r = r(MIXED_NEW, MIXED_LEN) if r else wild_ranges(MIXED_NEW, MIXED_LEN, b.rng)
    run(b, MIXED_NEW, 2, ranges=r, slopes=slopes, window=window)
    few = [1, 3, 0, 2, 4, 3, 1, 1, 2, 2]
    run(b, few, 4, ranges=wild_ranges(few, MIXED_LEN, b.rng) if kind == "wild" else
        (prefix_ranges if kind == "prefix" else doc_ranges)(few, MIXED_LEN), slopes=slopes, window=window)
    b.cache.close()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows(pool, G, d):
    """Single tokens and a few: the sizes around 16 rows of a K/V head, short and long contexts."""
    lens = [1, 2, 7, 8, 9, 31, 33, 64, 127, 500, 1000, 1025]
    for B, m in ((8, 1), (16, 2), (32, max(1, 16 // G)), (16, 16 // G + 1)):
        b = Batch(pool, d, 2, B, [max(c, m) for c in lens], seed=G + m)
        run(b, [m] * len(lens), G)
        b.cache.close()


@pytest.mark.parametrize("pool", POOLS)
def test_one_long_context(pool):
    """One context split over many parts and joined."""
    b = Batch(pool, 128, 2, 16, [9001], seed=5)
    run(b, [1], 4)
    run(b, [3], 1, window=5000)
    run(b, [40], 2, cap=20.0, qmul=3.0)
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "fp8", "int4"])
@pytest.mark.parametrize("G", [1, 8])
def test_prompts_of_many_tiles(pool, G):
    b = Batch(pool, 128, 1, 16, [700, 1153], seed=G)
    run(b, [700, 900], G)
    b.cache.close()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("new", [[129, 40], [2, 1]])
def test_what_is_masked_never_reaches_a_row(pool, new):
    """NaN and infinite keys and values at positions that some rows see and others do not."""
    b = Batch(pool, 64, 2, 8, [200, 90], seed=9)
    spots = [(0, 150), (0, 199), (1, 60), (1, 88)]
    for s, p in spots:
        blk, off = b.tab[s][p // 8], p % 8
        if pool == "int4":
            b.k[blk, :, 0, 4 * 64 + off * 4:4 * 64 + off * 4 + 4] = O4.NAN_BYTE
            b.v[blk, :, 0, 4 * 64 + off::8] = O4.NAN_BYTE
        elif pool == "fp8":
            b.k[blk, :, off], b.v[blk, :, off] = 0x7F, 0x7F
        else:
            b.k[blk, :, off], b.v[blk, :, off] = np.nan, np.inf if p % 2 else np.nan
    b.upload()
    got, q, _ = run(b, new, 2, check=False)
    at = 0
    for s, m in enumerate(new):
        k, v = b.values(s, "k"), b.values(s, "v")
        c = b.lens[s]
        for i in range(m):
            p = c - m + i
            if any(t == s and x <= p for t, x in spots):
                assert np.isnan(got[at + i]).all(), (s, i)
                continue
            want = OQ.query_attention(q[at + i:at + i + 1], k[:p + 1], v[:p + 1], 0.125)
            tol = tolerance(pool, q[at + i:at + i + 1].astype(np.float64), k[:p + 1], v[:p + 1], 20.0, 0.125, 0.0, want)
            close(got[at + i:at + i + 1], want, tol, (s, i))
        at += m
    b.cache.close()


def test_large_and_extreme_scores():
    """Scores of thousands (one weight takes all), of either sign, and values near float16's limits."""
    b = Batch("f16", 128, 2, 16, [300, 77], seed=2)
    for new in ([300, 60], [1, 2]):
        run(b, new, 2, scale=20.0)
        run(b, new, 2, scale=1e-6)
        run(b, new, 2, scale=3.0, cap=1000.0, qmul=8.0)
    b.v = (b.v.astype(np.float32) * 10000).clip(-65504, 65504).astype(np.float16)
    b.upload()
    run(b, [300, 60], 2)
    run(b, [1, 2], 2)
    b.cache.close()


def test_fp8_scales_of_any_size():
    for lo, hi in ((1e-6, 2e-6), (50.0, 200.0), (1e-4, 10.0)):
        b = Batch("fp8", 128, 1, 8, [260, 50], seed=4, vscale=(lo, hi))
        b.vs[::5] = 0.0
        b.upload()
        for new in ([200, 50], [1, 4]):
            got, q, _ = run(b, new, 4, check=False)
            at = 0
            for s, m in enumerate(new):
                want = OQ.query_attention(q[at:at + m], b.values(s, "k"), b.values(s, "v"), 1 / math.sqrt(128))
                tol = tolerance("fp8", q[at:at + m].astype(np.float64), b.values(s, "k"), b.values(s, "v"), 30.0,
                                1 / math.sqrt(128), 0.0, want)
                close(got[at:at + m], want, tol, (lo, s, m))
                at += m
        b.cache.close()


def test_released_blocks_are_not_read():
    """Entries of blocks wholly before the window, or outside every row's range, may be -1."""
    b = Batch("f16", 128, 2, 16, [500, 333], seed=6)
    tab = b.tab.copy()
    for new in ([40, 3], [1, 2]):
        b.tab = tab.copy()
        for s, m in enumerate(new):
            b.tab[s, :max(0, b.lens[s] - m - 63) // 16] = -1
        keep, b.tab = b.tab, tab
        want = run(b, new, 2, window=64, check=False)
        b.tab = keep
        got = run(b, new, 2, window=64, check=False, q_in=want[1])
        assert np.array_equal(got[0], want[0])
    b.cache.close()


def call(b, new_start, n, lens=None, max_queries=None, max_context=None, tab=None, G=1, **kw):
    q = torch.randn(n, b.H * G, b.d, device="cuda").half()
    out = torch.full_like(q, 7.5)
    up = lambda x: torch.tensor(np.asarray(x, dtype=np.int32)).cuda()       # noqa: E731
    b.cache.query_attention(0, q, up(new_start), up(b.tab if tab is None else tab), up(b.lens if lens is None else lens),
                            n if max_queries is None else max_queries,
                            max(b.lens) if max_context is None else max_context, 0.1, out=out, **kw)
    return q, out.cpu().numpy()


@pytest.mark.parametrize("big", [False, True])
def test_device_errors(big):
    """Bad lengths, rows and block ids are reported, and nothing outside the sequence's own rows is written."""
    n = 40 if big else 4
    b = Batch("f16", 128, 1, 16, [100, 60], seed=8)
    _, out = call(b, [0, n, 2 * n], 2 * n)
    assert b.cache.device_error() == 0 and (out != 7.5).any(-1).all()
    # rows out of order, beyond q, more than max_queries: the sequence is left out, the other is not
    for starts, mq in (([0, n, n - 1], n), ([0, n, 2 * n + 1], 2 * n), ([0, n, 2 * n], n - 1), ([-1, n, 2 * n], 2 * n)):
        _, out = call(b, starts, 2 * n, max_queries=mq)
        assert b.cache.device_error() == abi.KV_DEVERR_QUERY
        if starts[0] == 0 and mq >= n:
            assert (out[:n] != 7.5).any(-1).all() and (out[n:] == 7.5).all()
        elif starts[0] < 0:
            assert (out[:n] == 7.5).all() and (out[n:] != 7.5).any(-1).all()
        else:
            assert (out == 7.5).all()
    # a longer length than the bound is clamped; fewer cached tokens than rows: rows before position 0 are 0
    _, out = call(b, [0, n, 2 * n], 2 * n, max_context=90)
    assert b.cache.device_error() == abi.KV_DEVERR_CONTEXT and np.isfinite(out).all()
    _, out = call(b, [0, n, 2 * n], 2 * n, lens=[100, n - 3])
    assert b.cache.device_error() == abi.KV_DEVERR_CONTEXT and not out[n:n + 3].any() and out[n + 3:].any(-1).all()
    _, out = call(b, [0, n, 2 * n], 2 * n, lens=[-4, 60])
    assert b.cache.device_error() == abi.KV_DEVERR_CONTEXT and not out[:n].any()
    # a bad block id: reported, and read as block 0
    for bad in (-1, b.cache.num_blocks, 2 ** 31 - 1, -2 ** 31):
        tab = b.tab.copy()
        tab[1, 1] = bad
        call(b, [0, n, 2 * n], 2 * n, tab=tab)
        assert b.cache.device_error() == abi.KV_DEVERR_BLOCK_ID
    b.cache.close()


def test_refusals_of_the_binding():
    b = Batch("f16", 64, 2, 8, [20])
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    st, tab, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 4], [[0, 1, 2]], [20]))
    ok = dict(layer=0, q=q, query_start=st, block_tables=tab, context_lens=ln, max_queries=4, max_context=20, scale=0.1)
    b.cache.query_attention(**ok)
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q=q.transpose(0, 1)), dict(query_start=st.long()),
                dict(query_start=st[:1]), dict(context_lens=ln.long()), dict(block_tables=tab[0]), dict(out=q[:3]),
                dict(out=q.float()), dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(2)),
                dict(ranges=torch.zeros(4, 3, dtype=torch.int32, device="cuda")), dict(ranges=torch.zeros(4, 2, device="cuda")),
                dict(flags=abi.KV_DECODE_WORKSPACE_ZEROED), dict(block_tables=tab.cpu())):
        with pytest.raises(ValueError):
            b.cache.query_attention(**{**ok, **bad})
    for bad in (dict(scale=-1.0), dict(score_cap=float("nan")), dict(max_queries=5), dict(window=-1), dict(layer=1),
                dict(flags=8), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(abi.KvError) as e:
            b.cache.query_attention(**{**ok, **bad})
        assert e.value.status == abi.KV_ERR_INVALID_ARG
    assert b.cache.query_attention(**{**ok, "q": q[:0], "max_queries": 0}).shape == (0, 2, 64)
    b.cache.close()


@pytest.mark.parametrize("pool", ["f16", "int4"])
@pytest.mark.parametrize("new", [[1, 3], [200, 90]])
def test_streams_graphs_and_one_workspace(pool, new):
    """Another stream, a captured and replayed call, and calls one after the other on one zeroed workspace:
    the same bits."""
    b = Batch(pool, 128, 2, 16, [1500, 700], seed=1)
    want, q, _ = run(b, new, 4)
    side = torch.cuda.Stream()
    got = run(b, new, 4, stream=side, check=False, q_in=q)[0]
    assert np.array_equal(got, want)
    ws = b.cache.query_workspace(2, 8, max(new), 1500, num_tokens=sum(new))
    flags = abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL
    for _ in range(3):
        assert np.array_equal(run(b, new, 4, workspace=ws, flags=flags, check=False, q_in=q)[0], want)
    tq = torch.from_numpy(q).cuda()
    out = torch.zeros_like(tq)
    up = lambda x: torch.tensor(np.asarray(x, dtype=np.int32)).cuda()       # noqa: E731
    st, tab, ln = up(np.concatenate(([0], np.cumsum(new)))), up(b.tab), up(b.lens)
    for f in (flags, 0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                b.cache.query_attention(0, tq, st, tab, ln, max(new), 1500, 1 / math.sqrt(128), out=out, workspace=ws, flags=f)
        for _ in range(2):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(out.cpu().numpy(), want)
    # the queries change between replays: the new ones are read
    tq.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), run(b, new, 4, check=False, q_in=-q)[0])
    b.cache.close()


def test_offsets_beyond_4_gb():
    """Blocks of a pool far beyond 2^32 bytes."""
    B, H, d, nb = 16, 8, 128, 150_000                  # 4.9 GB each of K and V
    cache = PagedKVCache(1, nb, B, H, d, "f16")
    lens, ids = [100, 50], [[nb - 1, 7, nb - 3, 131072, 131071, 5, nb - 2], [nb - 4, nb - 9, 3, nb // 2]]
    tab = np.full((2, 8), -1, dtype=np.int32)
    rng = np.random.default_rng(0)
    kv = {}
    for s, c in enumerate(lens):
        tab[s, :len(ids[s])] = ids[s]
        for w, pool in (("k", cache.k[0]), ("v", cache.v[0])):
            x = rng.standard_normal((len(ids[s]) * B, H, d)).astype(np.float16)
            kv[s, w] = x[:c].astype(np.float64)
            pool[torch.tensor(ids[s], device="cuda")] = torch.from_numpy(x).cuda().view(len(ids[s]), B, H, d).transpose(1, 2)
    up = lambda x: torch.tensor(np.asarray(x, dtype=np.int32)).cuda()       # noqa: E731
    for new in ([90, 50], [1, 2]):
        q = rng.standard_normal((sum(new), 2 * H, d)).astype(np.float16)
        got = cache.query_attention(0, torch.from_numpy(q).cuda(), up([0, new[0], sum(new)]), up(tab), up(lens), max(new),
                                    100, 0.09).cpu().numpy().astype(np.float64)
        at = 0
        for s, m in enumerate(new):
            want = OQ.query_attention(q[at:at + m], kv[s, "k"], kv[s, "v"], 0.09)
            tol = tolerance("f16", q[at:at + m].astype(np.float64), kv[s, "k"], kv[s, "v"], 30.0, 0.09, 0.0, want)
            close(got[at:at + m], want, tol, (s, m))
            at += m
    cache.close()
