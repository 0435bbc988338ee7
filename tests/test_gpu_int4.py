"""GPU: decode attention over 4-bit pools against the float64 oracle on the values the pool holds.

Tolerance, derived: with weights p_t and values v_t the result is sum p v / sum p.  A relative
error e in every weight moves it by at most 2 e max|v|.  The weights' errors are those of the
exponential (2 ulp: 2^-22) and of the score (float32 sums of exact products: at most 2^-23 of
sum |q||k| per addition, 136 additions, times scale; the query's odd elements are divided by 16
in float16, off by at most 2^-25 each below 2^-10), plus the float16 rounding of p: 2^-11 with 8
query heads per K/V head, 2^-22 with up to 4 (two float16 terms).  Sums over n tokens are float32:
one rounding per 16 tokens and partition, 2^-24 each, counted as (n/16 + 40) 2^-24."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import int4 as O4
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import BlockAllocator, PagedKVCache, rope_table

pytestmark = pytest.mark.gpu


def random_pool(rng, shape, d):
    a = rng.integers(0, 256, shape, dtype=np.uint8)
    a[..., 4 * d:] = rng.integers(80, 110, a[..., 4 * d:].shape)      # scales 2^-5 .. 0.9
    return a


def poison_unused(pools, tables, lens, B, d, start=None):
    """NaN scales in every slot no sequence attends to: they must never reach a result."""
    nb = pools[0].shape[0]
    used = np.zeros((nb, B), dtype=bool)
    for s, n in enumerate(lens):
        for p in range(start[s] if start else 0, n):
            used[tables[s][p // B], p % B] = True
    for b, o in zip(*np.nonzero(~used)):
        t = o % 8
        pools[0][b, :, o // 8, 4 * d + t * (d // 16):4 * d + (t + 1) * (d // 16)] = O4.NAN_BYTE
        pools[1][b, :, o // 8, 4 * d + t::8] = O4.NAN_BYTE


def build(rng, lens, H, d, B, window=0, layers=1):
    per = [-(-n // B) for n in lens]
    nb = sum(per) + 2
    perm = rng.permutation(nb).astype(np.int32)
    width = max(per + [1]) + 1
    tab = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(per):
        tab[s, :k] = perm[at:at + k]
        at += k
    cache = PagedKVCache(layers, nb, B, H, d, "int4")
    pools = [random_pool(rng, cache.k[0].shape, d) for _ in range(2)]
    return cache, tab, pools


def oracle(pools, tab, lens, q, B, d, scale, window=0):
    """float64 result and the tolerance of the module's docstring."""
    S, Hq, _ = q.shape
    H = pools[0].shape[1]
    G = Hq // H
    out, tol = np.zeros((S, Hq, d)), 0.0
    for s, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        pos = np.arange(lo, n)
        if not len(pos):
            continue
        k, v = (O4.token_values(p, w, d, tab[s][pos // B], pos % B) for p, w in zip(pools, "kv"))
        for j in range(Hq):
            qj = q[s, j].astype(np.float64)
            out[s, j] = OA.decode_attention_one(qj, k[:, j // G], v[:, j // G], scale)
            mag = np.max(np.abs(k[:, j // G]) @ np.abs(qj)) * scale
            e = 136 * 2.0 ** -23 * mag + 2.0 ** -22 + (2.0 ** -11 if G == 8 else 2.0 ** -22) + (n / 16 + 40) * 2.0 ** -24
            e += d * 2.0 ** -25 * np.max(np.abs(k)) * scale
            tol = max(tol, 2 * e * np.max(np.abs(v)))
    return out, tol


def to_cache(cache, pools, layer=0):
    cache.k[layer].copy_(torch.from_numpy(pools[0]))
    cache.v[layer].copy_(torch.from_numpy(pools[1]))


def check(lens, H, G, d, B, window=0, partition=0, seed=0, flags=0, out_f16=False):
    rng = np.random.default_rng(seed)
    cache, tab, pools = build(rng, lens, H, d, B)
    start = [max(0, n - window) if window else 0 for n in lens]
    for s, lo in enumerate(start):                    # blocks wholly before the window: released
        tab[s, :lo // B] = -1
    poison_unused(pools, tab, lens, B, d, start)
    to_cache(cache, pools)
    q = rng.standard_normal((len(lens), H * G, d)).astype(np.float16)
    scale = 1 / math.sqrt(d)
    want, tol = oracle(pools, tab, lens, q, B, d, scale, window)
    t = [torch.from_numpy(x).cuda() for x in (q, tab, np.array(lens, dtype=np.int32))]
    got = cache.attention_ex(0, *t, max(max(lens), 1), scale, window=window, partition_tokens=partition, flags=flags,
                             out_dtype=torch.float16 if out_f16 else torch.float32)
    assert cache.device_error() == 0
    err = np.abs(got.double().cpu().numpy() - want)
    if out_f16:
        tol = tol + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
    assert np.all(err <= tol), (float(err.max()), tol if np.isscalar(tol) else float(np.min(tol)))
    cache.close()


LENS = [0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 65, 100, 255, 256, 257, 300]


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("d,B,H", [(128, 16, 3), (128, 8, 2), (128, 32, 1), (64, 8, 2), (64, 16, 1), (64, 32, 3)])
def test_edges(G, d, B, H):
    check(LENS, H, G, d, B, seed=G + B)


@pytest.mark.parametrize("partition", [32, 64, 160])
@pytest.mark.parametrize("G,d", [(1, 128), (8, 128), (4, 64)])
def test_partitions(partition, G, d):
    """One- and two-level merges: up to 30 partitions."""
    check([957, 33, 0, 32, 640, 1], 2, G, d, 16, partition=partition, seed=partition)


@pytest.mark.parametrize("window", [1, 5, 32, 100, 1000])
@pytest.mark.parametrize("G,d,B", [(1, 128, 8), (8, 64, 32), (2, 128, 16)])
def test_window(window, G, d, B):
    check([0, 1, 6, 99, 100, 101, 777], 2, G, d, B, window=window, partition=64, seed=window)


@pytest.mark.parametrize("G,flags", [(1, 0), (8, abi.KV_DECODE_PDL)])
def test_more_sequences_than_one_launch_takes(G, flags):
    """1024 sequences go in one launch; the second starts at its own queries, tables, lengths and outputs."""
    lens = [(7 * s) % 90 for s in range(1030)]
    lens[3], lens[1027] = 700, 900
    check(lens, 1, G, 64, 16, flags=flags, seed=G)


def test_window_up_to_the_int_range():
    check([0, 5, 300], 1, 1, 128, 16, window=2 ** 31 - 1)


def test_float16_output_and_long_context():
    check([5000, 17], 2, 1, 128, 16, out_f16=True, seed=3)
    check([3001, 900, 0], 1, 8, 128, 32, out_f16=True, seed=4)
    check([20011], 1, 1, 64, 8, seed=5)


def test_more_sequences_than_a_launch_takes():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 40, 2100).tolist()
    check(lens, 1, 2, 64, 8, seed=6)


def test_large_scores_and_equal_keys():
    """Scores far above the lazy maximum's slack, increasing along the context, and constant values."""
    rng = np.random.default_rng(7)
    lens, H, d, B = [300], 1, 128, 16
    cache, tab, pools = build(rng, lens, H, d, B)
    k = np.linspace(0.01, 3, 300)[:, None, None] * np.ones((300, 1, d))
    v = rng.standard_normal((300, 1, d))
    for w, x, p in (("k", k, pools[0]), ("v", v, pools[1])):
        c, s = O4.quantize(x.astype(np.float32))
        for i in range(300):
            O4.store(p, w, tab[0][i // B], 0, i % B, c[i, 0], s[i, 0])
    to_cache(cache, pools)
    q = np.full((1, 1, d), 4.0, dtype=np.float16)
    want, tol = oracle(pools, tab, lens, q, B, d, 1.0)
    got = cache.attention_ex(0, *(torch.from_numpy(x).cuda() for x in (q, tab, np.array(lens, dtype=np.int32))), 300, 1.0)
    assert np.max(np.abs(got.double().cpu().numpy() - want)) <= tol
    cache.close()


@pytest.mark.parametrize("in_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("G,d,B", [(1, 128, 16), (4, 64, 8), (8, 128, 32)])
def test_fused_append_equals_append_then_attend(in_dtype, G, d, B):
    rng = np.random.default_rng(8)
    lens, H = [1, 8, 9, 33, 500, 0, 16], 2
    cache, tab, pools = build(rng, lens, H, d, B)
    poison_unused(pools, tab, [max(n - 1, 0) for n in lens], B, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), H * G, d)).astype(np.float16)).cuda()
    kn, vn = (torch.from_numpy(rng.standard_normal((len(lens), H, d)).astype(np.float32)).cuda().to(in_dtype) for _ in range(2))
    tabs, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    results = []
    for fused in (True, False):
        to_cache(cache, pools)
        if fused:
            out = cache.attention_ex(0, q, tabs, ln, 500, 0.1, k_new=kn, v_new=vn, partition_tokens=64)
        else:
            slots = torch.tensor([tab[s][(n - 1) // B] * B + (n - 1) % B if n else -1 for s, n in enumerate(lens)], device="cuda")
            cache.append(0, kn, vn, slots)
            out = cache.attention_ex(0, q, tabs, ln, 500, 0.1, partition_tokens=64)
        results.append((out.clone(), cache.k[0].clone(), cache.v[0].clone()))
    assert cache.device_error() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
    pools = [results[1][1].cpu().numpy(), results[1][2].cpu().numpy()]
    want, tol = oracle(pools, tab, lens, q.cpu().numpy(), B, d, 0.1)
    assert np.max(np.abs(results[0][0].double().cpu().numpy() - want)) <= tol
    cache.close()


def test_every_entry_point_gives_the_same():
    rng = np.random.default_rng(9)
    lens, H, d, B = [70, 300, 12], 2, 128, 16
    cache, tab, pools = build(rng, lens, H, d, B)
    to_cache(cache, pools)
    q = torch.from_numpy(rng.standard_normal((3, H, d)).astype(np.float16)).cuda()
    tabs, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    base = cache.attention(0, q, tabs, ln, 300, 0.1)
    assert torch.equal(cache.attention_gqa(0, q, tabs, ln, 300, 0.1), base)
    assert torch.equal(cache.attention_ex(0, q, tabs, ln, 300, 0.1), base)
    out = torch.zeros_like(base)
    abi.paged_decode_attention_static(cache.handle, 0, q.data_ptr(), out.data_ptr(), tabs.data_ptr(), tabs.shape[1],
                                      ln.data_ptr(), 3, 300, 0.1, 0, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, base)
    kn = torch.randn(3, H, d, device="cuda").half()
    a = cache.attention_append(0, q, kn, kn, tabs, ln, 300, 0.1)
    assert torch.equal(cache.attention(0, q, tabs, ln, 300, 0.1), a)
    assert abi.kv_pool_features(cache.handle) == 0
    cache.close()


def test_flags_repeat_capture_and_two_streams():
    """A kept zeroed workspace over several calls, all launch flags, a captured graph and a second
    graph on its own workspace and stream: always the plain call's bits."""
    rng = np.random.default_rng(10)
    lens, H, d, B = [900, 40, 1, 333], 4, 128, 16
    cache, tab, pools = build(rng, lens, H, d, B)
    to_cache(cache, pools)
    q = torch.from_numpy(rng.standard_normal((4, H, d)).astype(np.float16)).cuda()
    tabs, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    base = cache.attention_ex(0, q, tabs, ln, 900, 0.1, partition_tokens=64)
    fl = abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL | abi.KV_DECODE_EARLY_TABLES | abi.KV_DECODE_EARLY_POOL
    ws = [cache.zeroed_workspace(4, 900, partition_tokens=64) for _ in range(2)]
    outs = [torch.zeros_like(base) for _ in range(2)]
    for _ in range(4):
        cache.attention_ex(0, q, tabs, ln, 900, 0.1, partition_tokens=64, flags=fl, workspace=ws[0], out=outs[0])
        assert torch.equal(outs[0], base)
    counters = abi.paged_decode_workspace_size(cache.handle, 4, 900, 64)
    assert counters <= ws[0].numel() and int(ws[0][:512].sum()) == 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        streams[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            for _ in range(3):
                cache.attention_ex(0, q, tabs, ln, 900, 0.1, partition_tokens=64, flags=fl, workspace=ws[i],
                                   out=outs[i], stream=streams[i])
    torch.cuda.synchronize()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], base) and torch.equal(outs[1], base)
    assert cache.device_error() == 0
    cache.close()


def test_bad_tables_and_lengths_are_flagged():
    rng = np.random.default_rng(11)
    lens, H, d, B = [40, 20], 1, 64, 8
    cache, tab, pools = build(rng, lens, H, d, B)
    to_cache(cache, pools)
    q = torch.zeros(2, 1, d, device="cuda").half()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bad = tab.copy()
    bad[1, 1] = cache.num_blocks
    good = cache.attention(0, q, torch.from_numpy(tab).cuda(), ln, 40, 0.1).clone()
    out = cache.attention(0, q, torch.from_numpy(bad).cuda(), ln, 40, 0.1)
    assert cache.device_error() == abi.KV_DEVERR_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.isfinite(out).all()
    # a fused append whose block id is bad stores nothing
    before = [cache.k[0].clone(), cache.v[0].clone()]
    bad[1, 1], bad[1, 2] = tab[1, 1], -7
    kn = torch.ones(2, 1, d, device="cuda").half()
    cache.attention_append(0, q, kn, kn, torch.from_numpy(bad).cuda(), ln, 40, 0.1)
    assert cache.device_error() == abi.KV_DEVERR_BLOCK_ID
    last = int(tab[0, 39 // B])
    for t, b4 in zip((cache.k[0], cache.v[0]), before):
        changed = (t != b4).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed in ([], [last])                 # only the other sequence's block
        t.copy_(b4)
    long = torch.tensor([41, -1], dtype=torch.int32, device="cuda")
    out = cache.attention(0, q, torch.from_numpy(tab).cuda(), long, 40, 0.1)
    assert cache.device_error() == abi.KV_DEVERR_CONTEXT
    assert torch.equal(out[0], good[0]) and torch.all(out[1] == 0)
    cache.close()


def test_copy_blocks_and_swap():
    rng = np.random.default_rng(12)
    cache = PagedKVCache(2, 6, 16, 3, 64, "int4")
    host = []
    for t in cache.k + cache.v:
        a = rng.integers(0, 256, t.shape, dtype=np.uint8)
        t.copy_(torch.from_numpy(a))
        host.append(a)
    cache.copy_blocks(torch.tensor([[1, 4]], dtype=torch.int32, device="cuda"))
    blocks = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    image = cache.swap_out(blocks)
    cache.swap_in(image, torch.tensor([5, 2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for t, a in zip(cache.k + cache.v, host):
        a[4], a[5], a[2] = a[1].copy(), a[0].copy(), a[1].copy()
        assert np.array_equal(t.cpu().numpy(), a)
    assert cache.device_error() == 0
    cache.close()


@pytest.mark.parametrize("G", [1, 8])
def test_prompt_decode_and_read_back_together(G):
    """A served batch: two prompts rotated and appended, decode steps that rotate, append and
    attend through the allocator's tables, one forked candidate with copy-on-write, and the cache
    read back, against the oracle on the float32 rotation's quantised values."""
    from oracle import rope as OR
    rng = np.random.default_rng(13)
    H, d, B, steps = 2, 128, 16, 5
    scale = 1 / math.sqrt(d)
    cache = PagedKVCache(1, 40, B, H, d, "int4")
    for t in cache.k + cache.v:
        t.fill_(0xFF)
    alloc = BlockAllocator(40, B, rng.permutation(40))
    tab = rope_table(512, d, 10000.0)
    table = tab.cpu().numpy()
    model = {}                                          # sequence -> (k, v) float64 rows the cache must hold

    def rows(n):
        return (rng.standard_normal((n, h, d)).astype(np.float16) for h in (H * G, H, H))

    def feed(ids, counts):
        """Append counts[i] tokens to ids[i] in one call; returns the rotated queries (host)."""
        slots, pos, pairs = [], [], []
        for s, c in zip(ids, counts):
            n0 = alloc.seq_info(s)[0]
            sl, cow = alloc.append_slots(s, c)
            if cow:
                pairs.append(cow)
            slots += sl
            pos += range(n0, n0 + c)
        if pairs:
            cache.copy_blocks(torch.tensor(pairs, dtype=torch.int32, device="cuda"))
        q, k, v = rows(len(slots))
        pos = np.array(pos, dtype=np.int32)
        q_out = cache.append_rope(0, *(torch.from_numpy(x).cuda() for x in (k, v, np.array(slots, dtype=np.int64), pos)),
                                  tab, q=torch.from_numpy(q).cuda())
        rk = OR.rotate(k, table[pos], d, False, np.float32)
        rv = v.astype(np.float32)
        at = 0
        for s, c in zip(ids, counts):
            new = [O4.dequantize(*O4.quantize(x[at:at + c])) for x in (rk, rv)]
            old = model.get(s, [np.zeros((0, H, d))] * 2)
            model[s] = [np.concatenate([a, b]) for a, b in zip(old, new)]
            at += c
        return q_out

    a, b = alloc.new_seq(), alloc.new_seq()
    feed([a, b], [37, 90])
    c = alloc.fork(a)
    model[c] = list(model[a])
    ids = [a, b, c]
    for _ in range(steps):
        q = feed(ids, [1, 1, 1])
        tabs, lens = alloc.build_tables(ids, 8)
        out = cache.attention_ex(0, q, torch.tensor(tabs, dtype=torch.int32, device="cuda"),
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), scale)
        qh = q.cpu().numpy()
        pools = [cache.k[0].cpu().numpy(), cache.v[0].cpu().numpy()]
        want, tol = oracle(pools, np.array(tabs), lens, qh, B, d, scale)
        assert np.max(np.abs(out.double().cpu().numpy() - want)) <= tol
        for s, n in zip(ids, lens):
            assert model[s][0].shape[0] == n
    for s in ids:
        n = alloc.seq_info(s)[0]
        t = alloc.table(s)
        slots = torch.tensor([t[p // B] * B + p % B for p in range(n)], device="cuda")
        k, v = cache.gather(0, slots)
        assert np.array_equal(k.double().cpu().numpy(), model[s][0])
        assert np.array_equal(v.double().cpu().numpy(), model[s][1])
    assert cache.device_error() == 0
    cache.close()


def test_decode_step_in_one_call():
    """kv_decode_step over a 4-bit pool (slot reservation, copy-on-write of a forked block, copies,
    fused append and attention) against append_rope-free steps made call by call: same bits."""
    import ctypes
    H, d, B, prompt, cands, steps = 3, 128, 16, 37, 3, 6
    runs = []
    for one_call in (True, False):
        rng = np.random.default_rng(14)
        cache = PagedKVCache(1, 32, B, H, d, "int4")
        for t in cache.k + cache.v:
            t.fill_(0xFF)
        alloc = BlockAllocator(32, B, rng.permutation(32))
        root = alloc.new_seq()
        slots, _ = alloc.append_slots(root, prompt)
        pk, pv = (torch.from_numpy(rng.standard_normal((prompt, H, d)).astype(np.float16)).cuda() for _ in range(2))
        cache.append(0, pk, pv, torch.tensor(slots, device="cuda"))
        seqs = [root] + [alloc.fork(root) for _ in range(cands - 1)]
        nb = -(-(prompt + steps) // B)
        width = cands * nb + 3 * cands
        meta = torch.empty(width, dtype=torch.int32, device="cuda")
        x = torch.empty(3, cands, H, d, dtype=torch.float16, device="cuda")
        out = torch.empty(cands, H, d, device="cuda")
        ws = cache.zeroed_workspace(cands, prompt + steps)
        outs = []
        for _ in range(steps):
            new = torch.from_numpy(rng.standard_normal((3, cands, H, d)).astype(np.float16)).pin_memory()
            if one_call:
                a = abi.kv_decode_args()
                a.q, a.k_new, a.v_new, a.in_dtype = x[0].data_ptr(), x[1].data_ptr(), x[2].data_ptr(), abi.KV_F16
                a.out, a.block_tables, a.max_blocks_per_seq = out.data_ptr(), meta.data_ptr(), nb
                a.context_lens, a.batch, a.max_context = meta.data_ptr() + 4 * cands * nb, cands, prompt + steps
                a.scale, a.workspace, a.workspace_bytes = 0.1, ws.data_ptr(), ws.numel()
                a.stream = torch.cuda.current_stream().cuda_stream
                a.flags = abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL
                staging = torch.empty(width, dtype=torch.int32).pin_memory()
                back = torch.empty(cands, H, d).pin_memory()
                abi.kv_decode_step(alloc.handle, cache.handle, (ctypes.c_int32 * cands)(*seqs), cands, nb,
                                   staging.data_ptr(), meta.data_ptr(), new.data_ptr(), x.data_ptr(), x.numel() * 2,
                                   back.data_ptr(), out.numel() * 4, a)
                torch.cuda.synchronize()
                outs.append(back.clone())
            else:
                slots, pairs = [], []
                for s in seqs:
                    sl, cow = alloc.append_slots(s, 1)
                    slots += sl
                    pairs += [cow] if cow else []
                if pairs:
                    cache.copy_blocks(torch.tensor(pairs, dtype=torch.int32, device="cuda"))
                q, k, v = new.cuda()
                cache.append(0, k, v, torch.tensor(slots, device="cuda"))
                tabs, lens = alloc.build_tables(seqs, nb)
                outs.append(cache.attention(0, q, torch.tensor(tabs, dtype=torch.int32, device="cuda"),
                                            torch.tensor(lens, dtype=torch.int32, device="cuda"), prompt + steps, 0.1).cpu())
        assert cache.device_error() == 0
        runs.append((torch.stack(outs), cache.k[0].cpu(), cache.v[0].cpu()))
        cache.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_blocks_beyond_four_gigabytes():
    """Slots whose byte offset in the pool needs more than 32 bits: append, read back and attend."""
    B, H, d = 16, 40, 128
    nb = 100_000                                        # 4.6 GB each of K and V
    cache = PagedKVCache(1, nb, B, H, d, "int4")
    rng = np.random.default_rng(15)
    n = 50
    tab = np.array([[nb - 1, 3, nb - 5, 93_207]], dtype=np.int32)
    slots = np.array([tab[0][p // B] * B + p % B for p in range(n)], dtype=np.int64)
    k, v = (rng.standard_normal((n, H, d)).astype(np.float16) for _ in range(2))
    cache.append(0, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.from_numpy(slots).cuda())
    kb, vb = cache.gather(0, torch.from_numpy(slots).cuda())
    kv = [O4.dequantize(*O4.quantize(x)) for x in (k, v)]
    assert np.array_equal(kb.double().cpu().numpy(), kv[0]) and np.array_equal(vb.double().cpu().numpy(), kv[1])
    q = rng.standard_normal((1, H, d)).astype(np.float16)
    out = cache.attention(0, torch.from_numpy(q).cuda(), torch.from_numpy(tab).cuda(),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), n, 0.1)
    want = OA.decode_attention(q, [kv[0]], [kv[1]], 0.1)
    mag = max(np.max(np.abs(kv[0][:, h]) @ np.abs(q[0, h].astype(np.float64))) for h in range(H)) * 0.1
    e = 136 * 2.0 ** -23 * mag + 2.0 ** -21 + (n / 16 + 40) * 2.0 ** -24 + d * 2.0 ** -25 * np.max(np.abs(kv[0])) * 0.1
    assert np.max(np.abs(out.double().cpu().numpy() - want)) <= 2 * e * np.max(np.abs(kv[1]))
    assert cache.device_error() == 0
    cache.close()


@pytest.mark.parametrize("G,d", [(1, 128), (8, 128), (2, 64)])
def test_one_long_context_over_every_sm(G, d):
    """A single (sequence, head) cut into more ranges than a merge step joins, with and without
    whole units beside it, twice: the same bits, within the tolerance of the oracle."""
    rng = np.random.default_rng(16)
    lens, H, B = [40_003, 70, 0, 3000], 1, 32
    cache, tab, pools = build(rng, lens, H, d, B)
    to_cache(cache, pools)
    q = rng.standard_normal((len(lens), H * G, d)).astype(np.float16)
    want, tol = oracle(pools, tab, lens, q, B, d, 0.1)
    t = [torch.from_numpy(x).cuda() for x in (q, tab, np.array(lens, dtype=np.int32))]
    ws = cache.zeroed_workspace(len(lens), 50_000, num_q_heads=H * G)
    outs = [cache.attention_ex(0, *t, 50_000, 0.1, workspace=ws, flags=abi.KV_DECODE_WORKSPACE_ZEROED).clone()
            for _ in range(2)]
    assert torch.equal(outs[0], outs[1])
    assert np.max(np.abs(outs[0].double().cpu().numpy() - want)) <= tol
    assert cache.device_error() == 0
    cache.close()


def test_refusals():
    cache = PagedKVCache(1, 8, 16, 2, 128, "int4")
    q = torch.zeros(1, 6, 128, device="cuda").half()
    tab, ln = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(abi.KvError):                    # 3 query heads per K/V head
        cache.attention_gqa(0, q, tab, ln, 64, 0.1)
    for bad in (dict(partition_tokens=33), dict(partition_tokens=-32), dict(window=-1)):
        with pytest.raises(abi.KvError):
            cache.attention_ex(0, q[:, :2].contiguous(), tab, ln, 64, 0.1, **bad)
    groups = torch.tensor([[0, 2, 16]], dtype=torch.int32, device="cuda")
    with pytest.raises(abi.KvError):                    # prefix groups need an fp16 or FP8 pool
        cache.attention_ex(0, q[:1, :2].expand(2, 2, 128).contiguous(), tab.expand(2, 4).contiguous(), ln.expand(2).contiguous(),
                           64, 0.1, prefix_groups=groups)
    with pytest.raises(ValueError):
        PagedKVCache(1, 8, 16, 2, 128, "int3")
    with pytest.raises(abi.KvError):
        PagedKVCache(1, 8, 16, 2, 96, "int4")
    cache.close()
