"""Operators measured beside their plain forms.

  rope    rotate new queries and keys by their positions and write keys and values into a paged
          cache (fp16, FP8 or 4-bit pools)
  gather  read cached tokens back from a paged pool into contiguous rows, dequantised
  attend  single-token decode attention over a cache held in 4 bits

With ``own`` false every operator is computed by elementary torch operations; with ``own`` true
by the calls a user makes of ``paged_kv_cache_169_gb300``.

A 4-bit pool is uint8 [num_blocks][H][B/8][8*d/2 + 8*d/16]: per group of 8 tokens the codes, then
one scale byte for every 16 elements of a token (an unsigned float of 5 exponent and 3 mantissa
bits with float16's bias: byte << 7 is the scale as float16).  value = (nibble - 8) * scale.
K codes are [token][d/2] bytes (low nibble: the even element), K scales [token][d/16].  V codes
are 16-bit pieces of 4 elements of one token, [8 chunks of d/8][token/2][d/32][token%2], V scales
[d/16][token].
"""

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
IN_DTYPE = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's new tokens of a 7B-shaped layer: the call whose latency counts
        {"name": "rope_decode_7b", "op": "rope", "pool": "f16", "in": "f16", "n": 8, "q_heads": 32, "heads": 32,
         "d": 128, "rot": 128, "pairs": "half", "B": 16, "packed": False, "pad": 0, "prefill": False},
        # a long prompt of a grouped-query layer, q, k and v as views of one packed projection
        {"name": "rope_prefill_gqa70b", "op": "rope", "pool": "f16", "in": "f16", "n": 8192, "q_heads": 64,
         "heads": 8, "d": 128, "rot": 128, "pairs": "half", "B": 16, "packed": True, "pad": 0, "prefill": True},
        # an odd-sized prompt of a 13B-shaped layer into a 4-bit pool, and its cached values back
        {"name": "rope_prefill_int4_13b", "op": "rope", "pool": "int4", "in": "f16", "n": 4097, "q_heads": 40,
         "heads": 40, "d": 128, "rot": 128, "pairs": "half", "B": 16, "packed": False, "pad": 0, "prefill": True},
        # float32 projections, half of each head rotated in adjacent pairs, padding rows, FP8 pool
        {"name": "rope_partial_fp8", "op": "rope", "pool": "fp8", "in": "f32", "n": 1000, "q_heads": 10, "heads": 5,
         "d": 64, "rot": 32, "pairs": "adjacent", "B": 8, "packed": False, "pad": 7, "prefill": True},
        # a cached 16k-token prefix of 13B-shaped heads read back from a 4-bit pool
        {"name": "gather_int4_13b", "op": "gather", "pool": "int4", "out": "f16", "n": 16384, "heads": 40, "d": 128,
         "B": 16, "pad": 0},
        # a short odd prefix from an FP8 pool, as float32, with padding rows
        {"name": "gather_fp8_odd", "op": "gather", "pool": "fp8", "out": "f32", "n": 777, "heads": 5, "d": 64,
         "B": 8, "pad": 9},
        # the smallest decode step: two short contexts, the new token appended by the same call
        {"name": "attend_tiny_append", "op": "attend", "S": 2, "lo": 5, "hi": 37, "q_heads": 2, "heads": 2, "d": 64,
         "B": 8, "window": 0, "append": True, "even": False},
        # a small serving batch of a 7B-shaped layer
        {"name": "attend_7b", "op": "attend", "S": 8, "lo": 512, "hi": 2048, "q_heads": 32, "heads": 32, "d": 128,
         "B": 16, "window": 0, "append": False, "even": False},
        # one layer of the 13B-shaped full decode step
        {"name": "attend_13b", "op": "attend", "S": 48, "lo": 2048, "hi": 2048, "q_heads": 40, "heads": 40, "d": 128,
         "B": 16, "window": 0, "append": False, "even": True},
        # grouped queries: 64 query heads over 8 K/V heads
        {"name": "attend_gqa70b", "op": "attend", "S": 32, "lo": 4096, "hi": 4096, "q_heads": 64, "heads": 8,
         "d": 128, "B": 16, "window": 0, "append": False, "even": True},
        # two long contexts of 13B-shaped heads: one context split over many SMs
        {"name": "attend_long_13b", "op": "attend", "S": 2, "lo": 32768, "hi": 32768, "q_heads": 40, "heads": 40,
         "d": 128, "B": 16, "window": 0, "append": False, "even": True},
        # a ragged serving batch, context lengths log-uniform from 16 to 16384
        {"name": "attend_ragged", "op": "attend", "S": 256, "lo": 16, "hi": 16384, "q_heads": 32, "heads": 32,
         "d": 128, "B": 32, "window": 0, "append": False, "even": False},
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "gather", "attend", "attend", "attend"])
    d, B = rng.choice([64, 128, 128]), rng.choice([8, 16, 32])
    heads = rng.choice([1, 2, 3, 5, 8, 16, 32, 40])
    if op == "rope":
        pool = rng.choice(["f16", "fp8", "int4"])
        return {"op": op, "pool": pool, "in": "f16" if pool == "f16" else rng.choice(["f16", "f32"]),
                "n": _log(rng, 1, 4096), "q_heads": heads * rng.choice([1, 1, 2]), "heads": heads, "d": d,
                "rot": rng.choice([d, d, d // 2]), "pairs": rng.choice(["half", "adjacent"]), "B": B,
                "packed": rng.random() < 0.5, "pad": rng.choice([0, 0, 5]), "prefill": rng.random() < 0.5}
    if op == "gather":
        return {"op": op, "pool": rng.choice(["f16", "fp8", "int4"]), "out": rng.choice(["f16", "f32"]),
                "n": _log(rng, 1, 8192), "heads": heads, "d": d, "B": B, "pad": rng.choice([0, 0, 5])}
    group = rng.choice([1, 1, 2, 4, 8]) if heads <= 16 else 1
    S = _log(rng, 1, 64)
    hi = _log(rng, 16, min(32768, 200_000 // S))
    return {"op": op, "S": S, "lo": _log(rng, 1, hi), "hi": hi, "q_heads": heads * group, "heads": heads, "d": d,
            "B": B, "window": rng.choice([0, 0, 0, 100]), "append": rng.random() < 0.3, "even": False}


# ------------------------------------------------------------------------------------ 4-bit layout

def _k_codes(pool, d):
    """View of a 4-bit K pool's codes: [blocks, H, B/8, 8 tokens, d/2]."""
    return pool[..., :4 * d].unflatten(-1, (8, d // 2))


def _k_scales(pool, d):
    return pool[..., 4 * d:].unflatten(-1, (8, d // 16))


def _v_codes(pool, d):
    """View of a 4-bit V pool's codes: [blocks, H, B/8, 8 chunks, 4 token pairs, d/32, 2 tokens, 2 bytes]."""
    return pool[..., :4 * d].unflatten(-1, (8, 4, d // 32, 2, 2))


def _v_scales(pool, d):
    return pool[..., 4 * d:].unflatten(-1, (d // 16, 8))


def _nibbles(b):
    """Bytes [..., m] -> values -8..7 [..., 2m], low nibble first."""
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float() - 8.0


def _scale_value(b):
    """Scale bytes -> float32."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _read_k(pool, d, blk, off):
    """K of tokens (block, offset): float32 [n, H, d]."""
    c = _nibbles(_k_codes(pool, d)[blk, :, off // 8, off % 8])
    s = _scale_value(_k_scales(pool, d)[blk, :, off // 8, off % 8])
    return (c.unflatten(-1, (d // 16, 16)) * s[..., None]).flatten(-2)


def _read_v(pool, d, blk, off):
    o, r = off // 8, off % 8
    c = _nibbles(_v_codes(pool, d)[blk, :, o, :, r // 2, :, r % 2]).flatten(-3)
    s = _scale_value(_v_scales(pool, d)[blk, :, o, :, r])
    return (c.unflatten(-1, (d // 16, 16)) * s[..., None]).flatten(-2)


def _quantise(x):
    """float32 [n, H, d] -> (nibbles uint8 [n, H, d], scale bytes uint8 [n, H, d/16])."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    # a true division (by a scalar, a GPU multiplies by the rounded reciprocal and breaks ties);
    # the largest scale keeps values in float16
    s = (top / torch.full_like(top, 7.0)).clamp(max=896.0)
    bits = s.view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - ((127 - 15) << 3)
    byte = torch.where(s < 2.0 ** -14, torch.round(s * 2.0 ** 17).to(torch.int32), normal)
    v = _scale_value(byte.to(torch.uint8))
    q = torch.where(v[..., None] > 0, torch.round(g / v[..., None]).clamp(-7, 7), 0.0)
    return (q + 8).to(torch.uint8).flatten(-2), byte.to(torch.uint8)


def _write(kpool, vpool, k, v, d, blk, off):
    """Write tokens (float32 [n, H, d]) into a 4-bit pool."""
    o, r = off // 8, off % 8
    c, s = _quantise(k)
    _k_codes(kpool, d)[blk, :, o, r] = c[..., 0::2] | (c[..., 1::2] << 4)
    _k_scales(kpool, d)[blk, :, o, r] = s
    c, s = _quantise(v)
    c = (c[..., 0::2] | (c[..., 1::2] << 4)).unflatten(-1, (8, d // 32, 2))
    _v_codes(vpool, d)[blk, :, o, :, r // 2, :, r % 2] = c
    _v_scales(vpool, d)[blk, :, o, :, r] = s


# ------------------------------------------------------------------------------------ inputs

TABLE_LEN = 40960


def _lens(case, seed):
    """Context lengths of an attend case: all `hi` when even, else log-uniform in [lo, hi]."""
    rng = np.random.default_rng([seed, 3])
    if case["even"]:
        return [case["hi"]] * case["S"]
    u = rng.uniform(math.log(case["lo"]), math.log(case["hi"] + 1), case["S"])
    return np.clip(np.floor(np.exp(u)).astype(np.int64), case["lo"], case["hi"]).tolist()


def _pool_shape(pool, nb, H, B, d):
    if pool == "int4":
        return (nb, H, B // 8, 4 * d + d // 2), torch.uint8
    return (nb, H, B, d), {"f16": torch.float16, "fp8": torch.uint8}[pool]


def _filled(pool, nb, H, B, d, gen):
    """A pool tensor holding cached tokens ~ N(0, 1) (codes drawn directly)."""
    shape, dt = _pool_shape(pool, nb, H, B, d)
    t = torch.empty(shape, dtype=dt, device="cuda")
    for part in t.split(max(1, (1 << 27) // math.prod(shape[1:]))):
        x = torch.randn(part.shape, generator=gen, device="cuda")
        if pool == "f16":
            part.copy_(x)
        elif pool == "fp8":
            part.copy_((x * 110.0).clamp(-448, 448).to(F8).view(torch.uint8))
        else:
            y = torch.randn(part.shape, generator=gen, device="cuda")
            lo, hi = ((z * 3.7).round_().clamp_(-7, 7).add_(8).to(torch.uint8) for z in (x, y))
            part.copy_(lo | (hi << 4))
            # scales: a seventh of the largest of 16 normal values, about 0.25
            part[..., 4 * d:] = (96 + 3 * x[..., 4 * d:]).round_().clamp_(85, 107).to(torch.uint8)
    return t


def _cache(case, pool, nb):
    """The framework's cache over a pool of this case's shape (its tensors are .k[0] and .v[0])."""
    from paged_kv_cache_169_gb300.cache import PagedKVCache
    return PagedKVCache(1, nb, case["B"], case["heads"], case["d"], pool)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng([int(seed), 1])
    H, d, B = case["heads"], case["d"], case["B"]
    st = {"case": case}

    def pools(pool, nb, fill):
        """K and V tensors: the cache's own with `own`, else plain tensors of the same layout."""
        shape, dt = _pool_shape(pool, nb, H, B, d)
        st["cache"] = _cache(case, pool, nb) if own else None
        for i, name in enumerate(("k_pool", "v_pool")):
            t = (st["cache"].k[0], st["cache"].v[0])[i] if own else torch.empty(shape, dtype=dt, device="cuda")
            if fill:
                t.copy_(_filled(pool, nb, H, B, d, gen))
            else:
                t.zero_()
            st[name] = t
        if pool == "fp8":
            for i, name in enumerate(("k_scale", "v_scale")):
                sc = torch.rand(nb, generator=gen, device="cuda") * 0.004 + 0.008
                if own:
                    t = (st["cache"].k_scale[0], st["cache"].v_scale[0])[i]
                    t[:nb].copy_(sc)
                    sc = t[:nb]
                st[name] = sc

    if case["op"] == "attend":
        lens = _lens(case, seed)
        per = [-(-n // B) for n in lens]
        nb, width = sum(per) + 3, max(per)
        perm = rng.permutation(nb).astype(np.int32)
        tab = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(per):
            tab[s, :k] = perm[at:at + k]
            at += k
        pools("int4", nb, True)
        st["lens_host"], st["max"] = lens, case["hi"]
        st["tables"] = torch.from_numpy(tab).cuda()
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = torch.randn(len(lens), case["q_heads"], d, generator=gen, device="cuda").half()
        st["out"] = torch.zeros_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(d)
        if case["append"]:
            for name in ("k_new", "v_new"):
                st[name] = torch.randn(len(lens), H, d, generator=gen, device="cuda").half()
            last = torch.tensor([n - 1 for n in lens], device="cuda")
            st["slots"] = st["tables"].gather(1, (last // B)[:, None])[:, 0].long() * B + last % B
            st["k_back"], st["v_back"] = torch.zeros_like(st["k_new"]), torch.zeros_like(st["v_new"])
        if own:
            st["workspace"] = st["cache"].zeroed_workspace(len(lens), case["hi"], num_q_heads=case["q_heads"],
                                                           window=case["window"])
        return st

    n, pad = case["n"], case["pad"]
    nb = -(-n // B) + 5
    perm = rng.permutation(nb)
    tok = np.arange(n)
    # prefill and gather: a sequence's tokens fill whole blocks in order; decode: one token each, anywhere
    if case["op"] == "gather" or case["prefill"]:
        slots = perm[tok // B] * B + tok % B
    else:
        slots = rng.permutation(nb * B)[:n]
    if pad:
        slots[pad - 1::pad] = -1
    st["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
    if case["op"] == "gather":
        pools(case["pool"], nb, True)
        dt = IN_DTYPE[case["out"]]
        st["k_back"], st["v_back"] = (torch.zeros(n, H, d, dtype=dt, device="cuda") for _ in range(2))
        return st

    pools(case["pool"], nb, False)
    Hq, dt = case["q_heads"], IN_DTYPE[case["in"]]
    if case["packed"]:
        x = torch.randn(n, Hq + 2 * H, d, generator=gen, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        st["q"], st["k"], st["v"] = (torch.randn(n, h, d, generator=gen, device="cuda").to(dt) for h in (Hq, H, H))
    start = int(rng.integers(0, TABLE_LEN - n))
    pos = start + tok if case["prefill"] else rng.integers(0, TABLE_LEN, n)
    st["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    # the rotation table a program keeps: cosines then sines of each position's angles
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
    ang = torch.arange(TABLE_LEN, dtype=torch.float64, device="cuda")[:, None] * freq
    st["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float().contiguous()
    st["q_out"] = torch.zeros(n, Hq, d, dtype=torch.float16, device="cuda")
    if case["pool"] == "int4":
        st["k_back"], st["v_back"] = (torch.zeros(n, H, d, dtype=torch.float16, device="cuda") for _ in range(2))
    return st


# ------------------------------------------------------------------------------------ one pass

def _rotate(x, cos, sin, rot, pairs):
    """Rotate the first `rot` elements of each head; float32 in and out."""
    c, s = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_rope(st):
    case = st["case"]
    B, d, rot, pool = case["B"], case["d"], case["rot"], case["pool"]
    live = st["slots"] >= 0
    row = st["cos_sin"][st["positions"].long()]
    cos, sin = row[:, :rot // 2], row[:, rot // 2:]
    q = _rotate(st["q"].float(), cos, sin, rot, case["pairs"])
    st["q_out"].copy_(torch.where(live[:, None, None], q.half(), st["q_out"]))
    # a padding token stands for the first live one: the same values at the same place again
    src = torch.where(live, torch.arange(case["n"], device=live.device), live.int().argmax())
    blk, off = st["slots"][src] // B, st["slots"][src] % B
    k = _rotate(st["k"].float(), cos, sin, rot, case["pairs"])[src]
    v = st["v"].float()[src]
    if pool == "int4":
        _write(st["k_pool"], st["v_pool"], k, v, d, blk, off)
        return {"q": st["q_out"], **_plain_gather(st)}
    for name, x in (("k", k), ("v", v)):
        if pool == "fp8":
            x = (x / st[name + "_scale"][blk][:, None, None]).clamp(-448, 448).to(F8).view(torch.uint8)
        st[name + "_pool"][blk, :, off] = x if pool == "fp8" else x.half()
    return _pools_out(st)


def _pools_out(st):
    f8 = st["case"]["pool"] == "fp8"
    return {"q": st["q_out"], "k": st["k_pool"].view(F8) if f8 else st["k_pool"],
            "v": st["v_pool"].view(F8) if f8 else st["v_pool"]}


def _plain_gather(st):
    case = st["case"]
    B, d = case["B"], case["d"]
    pool = case.get("pool", "int4")
    live = (st["slots"] >= 0)[:, None, None]
    at = st["slots"].clamp(min=0)
    blk, off = at // B, at % B
    if pool == "int4":
        k, v = _read_k(st["k_pool"], d, blk, off), _read_v(st["v_pool"], d, blk, off)
    else:
        k, v = (st[n + "_pool"][blk, :, off] for n in "kv")
        if pool == "fp8":
            k, v = (x.view(F8).float() * st[n + "_scale"][blk][:, None, None] for x, n in ((k, "k"), (v, "v")))
    for name, x in (("k_back", k), ("v_back", v)):
        st[name].copy_(torch.where(live, x.to(st[name].dtype), st[name]))
    return {"k": st["k_back"], "v": st["v_back"]}


def _plain_attend(st):
    case = st["case"]
    B, d, H, S = case["B"], case["d"], case["heads"], case["S"]
    G = case["q_heads"] // H
    back = {}
    if case["append"]:
        at = st["slots"]
        _write(st["k_pool"], st["v_pool"], st["k_new"].float(), st["v_new"].float(), d, at // B, at % B)
        back = _plain_gather(st)
    T = sum(st["lens_host"])
    lens = st["lens"].long()
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), lens, output_size=T)
    pos = torch.arange(T, device="cuda") - (lens.cumsum(0) - lens)[seq]
    blk, off = st["tables"][seq, pos // B].long(), pos % B
    k = _read_k(st["k_pool"], d, blk, off)
    q = st["q"].float().view(S, H, G, d)
    x = (k[:, :, None] * q[seq]).sum(-1) * st["scale"]
    del k
    if case["window"]:
        x = torch.where((pos >= lens[seq] - case["window"])[:, None, None], x, -math.inf)
    top = torch.segment_reduce(x, "max", lengths=lens, axis=0, unsafe=True)
    p = torch.exp(x - top[seq])
    total = torch.segment_reduce(p, "sum", lengths=lens, axis=0, unsafe=True)
    v = _read_v(st["v_pool"], d, blk, off)
    o = torch.segment_reduce(p[..., None] * v[:, :, None], "sum", lengths=lens, axis=0, unsafe=True)
    st["out"].copy_((o / total[..., None]).flatten(1, 2))
    return {"out": st["out"], **back}


def _own(st):
    from paged_kv_cache_169_gb300 import abi
    case, cache = st["case"], st["cache"]
    if case["op"] == "gather":
        k, v = cache.gather(0, st["slots"], k_out=st["k_back"], v_out=st["v_back"])
        return {"k": k, "v": v}
    if case["op"] == "rope":
        cache.append_rope(0, st["k"], st["v"], st["slots"], st["positions"], st["cos_sin"], q=st["q"],
                          q_out=st["q_out"], adjacent_pairs=case["pairs"] == "adjacent")
        if case["pool"] == "int4":
            k, v = cache.gather(0, st["slots"], k_out=st["k_back"], v_out=st["v_back"])
            return {"q": st["q_out"], "k": k, "v": v}
        return _pools_out(st)
    more = {"k_new": st["k_new"], "v_new": st["v_new"]} if case["append"] else {}
    out = cache.attention_ex(0, st["q"], st["tables"], st["lens"], st["max"], st["scale"], window=case["window"],
                             out=st["out"], workspace=st["workspace"],
                             flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL | abi.KV_DECODE_EARLY_TABLES,
                             **more)
    if case["append"]:
        k, v = cache.gather(0, st["slots"], k_out=st["k_back"], v_out=st["v_back"])
        return {"out": out, "k": k, "v": v}
    return {"out": out}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "gather": _plain_gather, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ work

def _row_bytes(pool, d):
    """Bytes of one token of one head in a pool."""
    return {"f16": 2 * d, "fp8": d, "int4": d // 2 + d // 16}[pool]


def work(case):
    H, d, B = case["heads"], case["d"], case["B"]
    if case["op"] == "attend":
        # expected tokens: log-uniform lengths on [lo, hi] have the mean (hi - lo) / ln(hi / lo)
        lo, hi = case["lo"], case["hi"]
        mean = hi if case["even"] or lo == hi else (hi + 1 - lo) / math.log((hi + 1) / lo)
        read = min(mean, case["window"]) if case["window"] else mean
        T = case["S"] * read
        q = 4 * case["S"] * case["q_heads"] * d                     # q in, out
        new = case["S"] * H * (4 * d + 6 * _row_bytes("int4", d)) if case["append"] else 0
        return {"bytes": int(2 * T * H * _row_bytes("int4", d) + q + 4 * T / B + 4 * case["S"] + new),
                "flops": int(4 * T * case["q_heads"] * d)}
    n = case["n"] - (case["n"] // case["pad"] if case["pad"] else 0)
    if case["op"] == "gather":
        out = {"f16": 2, "f32": 4}[case["out"]]
        return {"bytes": 2 * n * H * (_row_bytes(case["pool"], d) + out * d) + 8 * case["n"],
                "flops": 2 * n * H * d}
    i = {"f16": 2, "f32": 4}[case["in"]]
    Hq = case["q_heads"]
    back = 2 * n * H * (_row_bytes("int4", d) + 2 * d) if case["pool"] == "int4" else 0
    table = 4 * case["rot"] * n
    return {"bytes": n * (Hq * d * (i + 2) + 2 * H * (i * d + _row_bytes(case["pool"], d))) + 12 * case["n"] + table +
            back, "flops": 3 * n * (Hq + H) * case["rot"] + 3 * n * 2 * H * d}


# ------------------------------------------------------------------------------------ 64 bits

def _float_of(byte):
    """Value of an unsigned 5-exponent 3-mantissa byte, from its definition."""
    e, m = (byte.long() >> 3).double(), (byte.long() & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e - 18))


def _token_values(pool, which, d, blk, off):
    """float64 [n, H, d] of the tokens' K ("k") or V ("v") in a 4-bit pool, element by element."""
    tile = pool[blk, :, off // 8]                                     # [n, H, 4d + d/2] bytes
    r, e = (off % 8)[:, None], torch.arange(d, device=pool.device)[None]
    if which == "k":
        byte = r * (d // 2) + e // 2
        scale = r * (d // 16) + e // 16
    else:
        chunk, i = e // (d // 8), e % (d // 8)
        piece = ((chunk * 4 + r // 2) * (d // 32) + i // 4) * 2 + r % 2
        byte = piece * 2 + (i % 4) // 2
        scale = (e // 16) * 8 + r
    b, s = (tile.gather(2, i[:, None].expand(-1, tile.shape[1], -1)) for i in (byte, 4 * d + scale))
    return ((b >> (4 * (e % 2)).to(torch.uint8)) & 15).double().sub_(8) * _float_of(s)


def _nearest4(x):
    """float64 [..., d] -> the values its 4-bit form stands for (groups of 16)."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1, keepdim=True)
    s = torch.clamp(top / torch.full_like(top, 7.0), max=896.0)       # a true division: ties matter
    ulp = torch.exp2(torch.clamp(torch.frexp(s).exponent - 4, min=-17).double())
    s = torch.round(s / ulp) * ulp                                    # 4 significant bits, halves to even
    c = torch.round(g / torch.where(s > 0, s, 1.0)).clamp(-7, 7)
    return (c * s).flatten(-2)


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    B, d, H = case["B"], case["d"], case["heads"]
    slots = st.get("slots")
    if case["op"] != "attend":
        live = torch.nonzero(slots >= 0)[:, 0]
        blk, off = slots[live] // B, slots[live] % B
    if case["op"] == "gather":
        out = {}
        for w in "kv":
            pool = st[w + "_pool"]
            if case["pool"] == "int4":
                x = _token_values(pool, w, d, blk, off)
            elif case["pool"] == "fp8":
                x = pool.view(F8).double()[blk, :, off] * st[w + "_scale"].double()[blk][:, None, None]
            else:
                x = pool.double()[blk, :, off]
            out[w] = torch.zeros(case["n"], H, d, dtype=torch.float64, device=x.device).index_copy_(0, live, x)
        return out
    if case["op"] == "rope":
        rot, out = case["rot"], {}
        row = st["cos_sin"][st["positions"].long()].double()
        z = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]
        i = torch.arange(rot // 2, device=z.device)
        a, b = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        for w in "qkv":
            x = st[w].double()
            if w != "v":
                y = torch.complex(x[..., a], x[..., b]) * z
                x = x.index_copy(2, a, y.real).index_copy(2, b, y.imag)
            x = x[live]
            if w == "q" or case["pool"] == "int4":
                x = x if w == "q" else _nearest4(x)
                out[w] = torch.zeros(case["n"], *x.shape[1:], dtype=torch.float64, device=x.device).index_copy_(0, live, x)
                continue
            if case["pool"] == "fp8":
                x = (x / st[w + "_scale"].double()[blk][:, None, None]).clamp(-448, 448)
            out[w] = torch.zeros(st[w + "_pool"].shape, dtype=torch.float64, device=x.device)
            out[w][blk, :, off] = x
        return out
    S, G = case["S"], case["q_heads"] // H
    out = torch.zeros(S, case["q_heads"], d, dtype=torch.float64, device=slots.device if slots is not None else "cuda")
    back = {w: torch.zeros(S, H, d, dtype=torch.float64, device=out.device) for w in "kv"}
    for s, n in enumerate(st["lens_host"]):
        pos = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device=out.device)
        blk = st["tables"][s].long()[pos // B]
        kv = {w: _token_values(st[w + "_pool"], w, d, blk, pos % B) for w in "kv"}
        if case["append"]:
            for w in "kv":
                back[w][s] = kv[w][-1] = _nearest4(st[w + "_new"][s].double())
        q = st["q"][s].double().view(H, G, d)
        p = torch.softmax(torch.matmul(q, kv["k"].permute(1, 2, 0)) * st["scale"], -1)
        out[s] = torch.matmul(p, kv["v"].transpose(0, 1)).view(-1, d)
    return {"out": out, **(back if case["append"] else {})}
