"""GPU: kv_append_rope, kv_rope_table, kv_gather and kv_append into 4-bit pools, against the oracle.

The rotation is float32 products and sums rounded one by one, which numpy repeats bit for bit, so
rotated keys and queries, and what is stored from them, are compared exactly; the same values are
compared with the float64 rotation within the bound of those roundings."""

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import int4 as O4
from oracle import rope as OR
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_table

pytestmark = pytest.mark.gpu

NP = {"f16": np.float16, "f32": np.float32}


def pool_bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def expected_pool(before, which, x, slots, B, pool, scales=None):
    """The pool tensor after storing x (float32 [n, H, d], already rotated) at the slots."""
    after = before.copy()
    codes = O4.quantize(x) if pool == "int4" else None
    for i, s in enumerate(slots):
        if s < 0:
            continue
        b, off = int(s) // B, int(s) % B
        for h in range(x.shape[1]):
            if pool == "int4":
                O4.store(after, which, b, h, off, codes[0][i, h], codes[1][i, h])
            elif pool == "fp8":
                after[b, h, off] = OF.quantize(x[i, h], scales[b])
            else:
                after[b, h, off] = x[i, h].astype(after.dtype)
    return after


def run_case(pool, in_dtype, d, rot, adjacent, B, n, H=3, Hq=5, packed=False, pad=(), seed=0, in_place=False,
             consecutive=False, table_len=300):
    rng = np.random.default_rng(seed)
    nb = -(-n // B) + 3
    cache = PagedKVCache(1, nb, B, H, d, pool)
    for t in cache.k + cache.v:                       # whatever lies there must stay but for the slots
        if t.dtype == torch.uint8:
            t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
        else:
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    sc = [None, None]
    if pool == "fp8":
        sc = [rng.uniform(0.004, 0.02, nb).astype(np.float32) for _ in range(2)]
        cache.k_scale[0][:nb].copy_(torch.from_numpy(sc[0]))
        cache.v_scale[0][:nb].copy_(torch.from_numpy(sc[1]))
    slots = (np.arange(n) + 3 if consecutive else rng.permutation(nb * B)[:n]).astype(np.int64)
    for i in pad:
        slots[i] = -1 - i
    pos = rng.integers(0, table_len, n).astype(np.int32)
    for i in pad:
        pos[i] = -5                                   # a padding token's position is not read
    tab = rng.standard_normal((table_len, rot)).astype(np.float32)   # any table: not only unit rows
    dt = NP[in_dtype]
    q, k, v = (rng.standard_normal((n, h, d)).astype(dt) for h in (Hq, H, H))
    if packed:
        x = torch.from_numpy(np.concatenate([q, k, v], 1)).cuda()
        tq, tk, tv = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        tq, tk, tv = (torch.from_numpy(a).cuda() for a in (q, k, v))
    out_dt = torch.float32 if pool == "f32" else torch.float16
    sentinel = torch.full((n, Hq, d), 9.5, dtype=out_dt, device="cuda")
    before = [pool_bytes(t).view(t.cpu().numpy().dtype).reshape(t.shape) for t in (cache.k[0], cache.v[0])]
    q_out = tq if in_place else sentinel
    got_q = cache.append_rope(0, tk, tv, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(),
                              torch.from_numpy(tab).cuda(), q=tq, q_out=q_out, adjacent_pairs=adjacent)
    assert got_q.data_ptr() == q_out.data_ptr()
    assert cache.device_error() == 0
    live = slots >= 0
    rows = tab[np.where(live, pos, 0)]
    rq = OR.rotate(q, rows, rot, adjacent, np.float32)
    rk = OR.rotate(k, rows, rot, adjacent, np.float32)
    want_q = np.where(live[:, None, None], rq.astype(NP["f32" if pool == "f32" else "f16"]),
                      q if in_place else np.asarray(9.5, dtype=NP["f32" if pool == "f32" else "f16"]))
    assert np.array_equal(got_q.cpu().numpy(), want_q)
    # within the float32 roundings of the exact rotation: each of the two products and the sum are
    # off by 2^-24 of |x c| + |y s| at most, and the store by half a step of its type
    exact = OR.rotate(q, rows, rot, adjacent)
    size = OR.rotate(np.abs(q), np.abs(rows) * np.where(np.arange(rot) < rot // 2, 1, -1), rot, adjacent)
    size = np.abs(size) + np.abs(OR.rotate(np.abs(q), np.abs(rows), rot, adjacent))
    half_step = 0.0 if pool == "f32" else 2.0 ** -11
    tol = np.abs(exact) * half_step + size * 2.0 ** -22 + 2.0 ** -25
    assert np.all(np.abs(got_q.double().cpu().numpy() - exact)[live] <= tol[live])
    for which, x, t, b4, s in (("k", rk, cache.k[0], before[0], sc[0]), ("v", v.astype(np.float32), cache.v[0], before[1], sc[1])):
        want = expected_pool(b4, which, x, slots, B, pool, s)
        assert np.array_equal(pool_bytes(t), want.view(np.uint8).reshape(pool_bytes(t).shape)), which
    cache.close()


@pytest.mark.parametrize("pool,in_dtype", [("f32", "f32"), ("f16", "f16"), ("fp8", "f16"), ("fp8", "f32"),
                                           ("int4", "f16"), ("int4", "f32")])
@pytest.mark.parametrize("d,rot,adjacent,B", [(128, 128, False, 16), (128, 64, True, 8), (128, 96, False, 32),
                                              (64, 64, False, 16), (64, 16, True, 32), (64, 48, True, 8),
                                              (64, 32, False, 8), (128, 16, False, 16)])
def test_rope_append_every_pool(pool, in_dtype, d, rot, adjacent, B):
    run_case(pool, in_dtype, d, rot, adjacent, B, n=13, pad=(4, 11), seed=d + rot + B)


@pytest.mark.parametrize("n", [1, 2, 3, 64, 701])
@pytest.mark.parametrize("pool", ["f16", "int4"])
def test_rope_append_lengths(n, pool):
    run_case(pool, "f16", 128, 128, False, 16, n=n, H=1, Hq=4, consecutive=True, packed=True, seed=n)
    run_case(pool, "f16", 64, 32, True, 8, n=n, H=5, Hq=1, seed=n, pad=(n - 1,) if n > 1 else ())


def test_rope_append_in_place_packed_and_all_padding():
    run_case("f16", "f16", 128, 128, False, 16, n=33, packed=True, in_place=True, pad=(0, 1, 7))
    run_case("f32", "f32", 64, 48, False, 8, n=9, packed=True, in_place=True)
    run_case("int4", "f16", 128, 64, True, 32, n=10, in_place=True, consecutive=True)
    run_case("int4", "f16", 128, 64, True, 32, n=6, pad=range(6))


def test_rope_append_without_queries_and_empty():
    cache = PagedKVCache(1, 4, 16, 2, 64, "f16")
    cache.k[0].zero_()
    k = torch.randn(3, 2, 64, device="cuda").half()
    tab = rope_table(10, 64)
    slots = torch.tensor([1, 2, 5], device="cuda")
    pos = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    assert cache.append_rope(0, k, k, slots, pos, tab) is None
    assert torch.equal(cache.k[0][0][:, [1, 2, 5]].transpose(0, 1), k)       # position 0: unchanged
    assert cache.append_rope(0, k[:0], k[:0], slots[:0], pos[:0], tab) is None
    cache.close()


def test_rope_append_bad_slot_and_position_skip_the_token():
    cache = PagedKVCache(1, 4, 16, 2, 64, "int4")
    for t in (cache.k[0], cache.v[0]):
        t.zero_()
    k = torch.ones(5, 2, 64, device="cuda").half()
    q = torch.ones(5, 4, 64, device="cuda").half()
    out = torch.full_like(q, 7.0)
    tab = rope_table(10, 64)
    slots = torch.tensor([3, 64, 5, 6, 1 << 40], device="cuda")
    pos = torch.tensor([0, 0, -1, 10, 0], dtype=torch.int32, device="cuda")
    cache.append_rope(0, k, k, slots, pos, tab, q=q, q_out=out)
    assert cache.device_error() == abi.KV_DEVERR_SLOT | abi.KV_DEVERR_POSITION
    assert torch.all(out[1:] == 7) and torch.all(out[0] == 1)
    kk, _ = cache.gather(0, torch.tensor([3, 5, 6, 4], device="cuda"))
    assert torch.allclose(kk[0].float(), torch.ones(2, 64, device="cuda"), rtol=2 ** -4)   # a scale is off by 2^-4 at most
    assert torch.all(kk[1:] == 0)
    k2, v2 = cache.gather(0, torch.tensor([64, -1], device="cuda"))
    assert cache.device_error() == abi.KV_DEVERR_SLOT
    assert torch.all(k2 == 0) and torch.all(v2 == 0)
    cache.close()


@pytest.mark.parametrize("in_dtype,d,B", [("f16", 128, 16), ("f32", 64, 8), ("f16", 64, 32)])
def test_int4_append_bit_exact_with_specials(in_dtype, d, B):
    rng = np.random.default_rng(5)
    nb, H, n = 5, 3, 37
    cache = PagedKVCache(1, nb, B, H, d, "int4")
    before = [rng.integers(0, 256, cache.k[0].shape, dtype=np.uint8) for _ in range(2)]
    cache.k[0].copy_(torch.from_numpy(before[0]))
    cache.v[0].copy_(torch.from_numpy(before[1]))
    slots = rng.permutation(nb * B)[:n].astype(np.int64)
    slots[5] = -1
    k, v = ((rng.standard_normal((n, H, d)) * np.exp2(rng.uniform(-12, 8, (n, H, 1)))).astype(NP[in_dtype]) for _ in range(2))
    for x in (k, v):
        x[0, 0, :] = 0
        x[1, 0, 3] = np.nan
        x[2, 0, 2], x[2, 0, 3] = np.inf, -np.inf
        x[3, 0, :16] = 60000
        x[4, 0, :16] = 3e-7
        x[6, 0, :16] = np.arange(16) * 0.5 - 3.5      # halves: ties to even
        x[6, 1, :16] = [7] * 8 + [0.5, 1.5, -2.5, 3.5, -0.5, 6.5, -6.5, 0]
    cache.append(0, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.from_numpy(slots).cuda())
    for which, x, t, b4 in (("k", k, cache.k[0], before[0]), ("v", v, cache.v[0], before[1])):
        want = expected_pool(b4, which, x.astype(np.float32), slots, B, "int4")
        got = t.cpu().numpy()
        bad = np.isnan(O4.SCALES[got[..., 4 * d:]])    # codes of a NaN group: any
        assert np.array_equal(got[..., 4 * d:], want[..., 4 * d:]), which
        # compare values: codes under a NaN scale are not defined
        live = slots >= 0
        b, o = slots[live] // B, slots[live] % B
        gv, wv = (O4.token_values(p, which, d, b, o) for p in (got, want))
        assert np.array_equal(gv, wv, equal_nan=True)
        assert bad.any()
    assert cache.device_error() == 0
    cache.close()


@pytest.mark.parametrize("in_dtype,d", [("f16", 128), ("f32", 64)])
def test_int4_small_groups_bit_exact(in_dtype, d):
    """Groups whose scale lies below 2^-14, where its grid is coarse: amax/7 rounds down by up to a third and
    the largest quotients have to be held at 7.  By kv_append, kv_append_rope and the fused decode step."""
    rng = np.random.default_rng(14)
    B, H, n = 16, 2, 120
    nb = n // B + 1
    top = np.linspace(0.2, 9.0, n * H * (d // 16)).reshape(n, H, d // 16, 1) * 7 * 2.0 ** -17
    k, v = ((np.where(rng.random((n, H, d // 16, 16)) < 0.3, rng.choice([-1.0, 1.0], (n, H, d // 16, 16)),
                      rng.uniform(-1, 1, (n, H, d // 16, 16))) * top).reshape(n, H, d).astype(NP[in_dtype])
            for _ in range(2))
    slots = np.arange(n, dtype=np.int64)
    tk, tv, ts = (torch.from_numpy(x).cuda() for x in (k, v, slots))
    caches = [PagedKVCache(1, nb, B, H, d, "int4") for _ in range(3)]
    for c in caches:
        c.k[0].zero_()
        c.v[0].zero_()
    caches[0].append(0, tk, tv, ts)
    caches[1].append_rope(0, tk, tv, ts, torch.zeros(n, dtype=torch.int32, device="cuda"), rope_table(4, d))
    q = torch.zeros(n, H, d, device="cuda").half()     # a sequence per token: lengths 1 .. 16 in its block
    tab = (ts // B).to(torch.int32).reshape(n, 1)
    ln = (ts % B + 1).to(torch.int32)
    caches[2].attention_ex(0, q, tab, ln, B, 0.1, k_new=tk, v_new=tv)
    for which, x in (("k", k), ("v", v)):
        zero = np.zeros(caches[0].k[0].shape, dtype=np.uint8)
        want = expected_pool(zero, which, x.astype(np.float32), slots, B, "int4")
        for c in caches:
            assert np.array_equal(getattr(c, which)[0].cpu().numpy(), want), which
    for c in caches:
        assert c.device_error() == 0
        c.close()


@pytest.mark.parametrize("pool,out", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("fp8", "f16"), ("fp8", "f32"),
                                      ("int4", "f16"), ("int4", "f32")])
@pytest.mark.parametrize("n,H,d,B", [(1, 1, 64, 8), (45, 3, 128, 16), (2, 40, 128, 32), (333, 5, 64, 8)])
def test_gather(pool, out, n, H, d, B):
    rng = np.random.default_rng(n)
    nb = 7
    cache = PagedKVCache(2, nb, B, H, d, pool)
    for t in cache.k + cache.v:
        if pool == "int4":                             # any bytes whose scales are finite
            a = rng.integers(0, 256, t.shape, dtype=np.uint8)
            a[..., 4 * d:] %= 199
            t.copy_(torch.from_numpy(a))
        elif pool == "fp8":
            t.copy_(torch.from_numpy((rng.integers(0, 2, t.shape) * 128 + rng.integers(0, 127, t.shape)).astype(np.uint8)))
        else:
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    if pool == "fp8":
        for t in cache.k_scale + cache.v_scale:
            t.copy_(torch.from_numpy(rng.uniform(0.01, 0.1, t.shape).astype(np.float32)))
    slots = rng.integers(0, nb * B, n).astype(np.int64)               # the same slot may come twice
    if n > 2:
        slots[n // 2] = -3
    dt = {"f16": torch.float16, "f32": torch.float32}[out]
    ko, vo = (torch.full((n, H, d), 2.5, dtype=dt, device="cuda") for _ in range(2))
    cache.gather(1, torch.from_numpy(slots).cuda(), k_out=ko, v_out=vo)
    assert cache.device_error() == 0
    live = slots >= 0
    b, o = slots[live] // B, slots[live] % B
    for which, got, t in (("k", ko, cache.k[1]), ("v", vo, cache.v[1])):
        a = t.cpu().numpy()
        if pool == "int4":
            x = O4.token_values(a, which, d, b, o)
        elif pool == "fp8":
            s = (cache.k_scale if which == "k" else cache.v_scale)[1].cpu().numpy()
            code = torch.from_numpy(a[b, :, o]).view(torch.float8_e4m3fn).float().numpy()
            x = code * s[b][:, None, None]             # one float32 rounding
        else:
            x = a[b, :, o]
        want = np.full((n, H, d), 2.5, dtype=NP[out])
        with np.errstate(over="ignore"):
            want[live] = x.astype(np.float32).astype(NP[out])
        assert np.array_equal(got.cpu().numpy(), want), which
    cache.close()


def test_rope_table_far_positions():
    """Each entry is the float64 cosine or sine rounded once (half a step, 2^-24 relative), at
    positions where a float32 angle would be off by far more; CUDA's double sincos and pow are off
    by at most 2 ulp of float64, whose effect on the angle at 2^17 is below 2^-33."""
    n, rot = 131072 + 7, 64
    t = rope_table(n, rot, 10000.0).double().cpu().numpy()
    pick = np.array([0, 1, 2, 1000, 65535, 131071, n - 1])
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = pick[:, None] * f
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.all(np.abs(t[pick] - want) <= np.abs(want) * 2.0 ** -24 + 2.0 ** -33)
    s = rope_table(100, 16, 500.0, position_scale=0.25).double().cpu().numpy()
    a = np.arange(100)[:, None] * 0.25 * 500.0 ** (-np.arange(0, 16, 2) / 16)
    assert np.all(np.abs(s - np.concatenate([np.cos(a), np.sin(a)], 1)) <= 2.0 ** -24)


def test_rope_append_on_another_stream_captured_and_pdl():
    """The call on a side stream, captured into a graph and replayed on new inputs, with
    KV_DECODE_PDL before a decode call: the same bytes as eager calls."""
    B, H, d, n = 16, 4, 128, 6
    caches = [PagedKVCache(1, 8, B, H, d, "int4") for _ in range(2)]
    for c in caches:
        for t in c.k + c.v:
            t.zero_()
    tab = rope_table(64, d)
    slots = torch.arange(n, device="cuda") * 17
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(n, H, d, device="cuda").half() for _ in range(3))
    o = [torch.zeros_like(q) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        caches[0].append_rope(0, k, v, slots, pos, tab, q=q, q_out=o[0], flags=abi.KV_DECODE_PDL, stream=side)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            caches[0].append_rope(0, k, v, slots, pos, tab, q=q, q_out=o[0], flags=abi.KV_DECODE_PDL, stream=side)
    torch.cuda.synchronize()
    for t in (q, k, v):
        t.mul_(-1.5)
    graph.replay()
    torch.cuda.synchronize()
    caches[1].append_rope(0, k, v, slots, pos, tab, q=q, q_out=o[1])
    assert torch.equal(o[0], o[1])
    assert torch.equal(caches[0].k[0], caches[1].k[0]) and torch.equal(caches[0].v[0], caches[1].v[0])


def test_python_refusals():
    cache = PagedKVCache(1, 4, 16, 2, 64, "f16")
    k = torch.zeros(3, 2, 64, device="cuda").half()
    slots, pos, tab = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), rope_table(4, 64)
    for bad in (dict(slot_mapping=slots.int()), dict(positions=pos.long()), dict(k=k[:2]), dict(k=k.float()),
                dict(positions=pos[:2]), dict(cos_sin=tab.half()), dict(q=k[:, :, :32]), dict(q=k.float()),
                dict(q_out=k), dict(q=k, q_out=k.float()), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(k=k.bfloat16(), v=k.bfloat16())):
        a = dict(k=k, v=k, slot_mapping=slots, positions=pos, cos_sin=tab)
        a.update(bad)
        with pytest.raises(ValueError):
            cache.append_rope(0, a.pop("k"), a.pop("v"), a.pop("slot_mapping"), a.pop("positions"), a.pop("cos_sin"), **a)
    with pytest.raises(ValueError):
        cache.gather(0, slots.int())
    with pytest.raises(ValueError):
        cache.gather(0, slots, k_out=k)
    with pytest.raises(ValueError):
        cache.gather(0, slots, out_dtype=torch.bfloat16)
    with pytest.raises(abi.KvError):
        cache.append_rope(0, k, k, slots, pos, rope_table(4, 128))          # more than the head
    with pytest.raises(abi.KvError):
        cache.append_rope(0, k[:1].expand(3, -1, -1), k, slots, pos, tab)   # rows of stride 0
    with pytest.raises(abi.KvError):
        cache.append_rope(0, k, k, slots, pos, tab, q=k, q_out=torch.empty_like(k[:1]).expand(3, -1, -1))
    cache.close()


def test_rope_and_gather_beyond_four_gigabytes():
    """fp16 slots whose byte offset needs more than 32 bits."""
    B, H, d, nb = 16, 40, 128, 30_000                  # 4.9 GB each of K and V
    cache = PagedKVCache(1, nb, B, H, d, "f16")
    slots = torch.tensor([nb * B - 1, 5, 27_001 * B + 3], device="cuda")
    pos = torch.tensor([0, 7, 19], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(3, H, d, device="cuda").half() for _ in range(2))
    tab = rope_table(20, d)
    cache.append_rope(0, k, v, slots, pos, tab)
    kb, vb = cache.gather(0, slots)
    want = OR.rotate(k.cpu().numpy(), tab.cpu().numpy()[pos.cpu().numpy()], d, False, np.float32).astype(np.float16)
    assert np.array_equal(kb.cpu().numpy(), want) and torch.equal(vb, v)
    assert cache.device_error() == 0
    cache.close()


def test_new_outputs_belong_to_the_stream_of_the_call():
    """Work queued on the current stream must not reach (as a late zero fill) what another stream gathers."""
    cache = PagedKVCache(1, 4, 16, 2, 64, "f16")
    k, v = (torch.randn(48, 2, 64, device="cuda").half() for _ in range(2))
    slots = torch.arange(48, device="cuda")
    cache.append(0, k, v, slots)
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        busy = (busy @ busy).clamp_(-1, 1)
    gk, gv = cache.gather(0, slots, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(gk, k) and torch.equal(gv, v)
    pos = torch.zeros(48, dtype=torch.int32, device="cuda")
    tab = rope_table(4, 64, stream=side)
    out = cache.append_rope(0, k, v, slots, pos, tab, q=k, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, k)
    cache.close()


def test_tensors_elsewhere_are_refused():
    cache = PagedKVCache(1, 4, 16, 2, 64, "int4")
    k = torch.randn(3, 2, 64, device="cuda").half()
    slots = torch.arange(3, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    tab = rope_table(4, 64)
    for at in range(6):
        x = [k, k, slots, pos, tab, k]
        x[at] = x[at].cpu()
        with pytest.raises(ValueError):
            cache.append_rope(0, *x[:5], q=x[5])
    with pytest.raises(ValueError):
        cache.append_rope(0, k, k, slots, pos, tab, q=k, q_out=k.cpu())
    for at in range(3):
        x = [slots, k.clone(), k.clone()]
        x[at] = x[at].cpu()
        with pytest.raises(ValueError):
            cache.gather(0, x[0], k_out=x[1], v_out=x[2])
    cache.close()
