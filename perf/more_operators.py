"""Operators of masked, capped and biased attention over a paged cache, beside their plain forms.

  query  attention of each sequence's newest tokens (one to thousands) over its paged cache, with
         a causal, prefix or document mask, a sliding window, scores capped by a tanh and a bias
         that grows with distance (fp16, FP8 or 4-bit pools)
  rope   rotate new queries and keys by positions with several axes (time, height, width) and
         write keys and values into a paged cache

With ``own`` false every operator is computed by elementary torch operations; with ``own`` true
by the calls a user makes of ``paged_kv_cache_169_gb300``.

query: token i of a sequence with n new tokens and context length c stands at position
p = c - n + i and sees the positions j of [first, last) (default: 0 and p + 1), less those before
p - window + 1.  With x = scale * q . k, the score is cap * tanh(x / cap) - slope * |p - j|; the
output is the softmax-weighted sum of the values, and 0 where nothing is seen.

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
TABLE_LEN = 40960


# ------------------------------------------------------------------------------------ cases

def _query(name, **k):
    c = {"name": name, "op": "query", "pool": "f16", "S": 1, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 0,
         "q_heads": 32, "heads": 32, "d": 128, "B": 16, "mask": "causal", "window": 0, "cap": 0.0, "slopes": False,
         "packed": False}
    c.update(k)
    return c


def listed():
    return [
        # the smallest call: two short prompts of a toy model, latency only
        _query("query_tiny", S=2, new_lo=5, new_hi=37, q_heads=2, heads=2, d=64),
        # four 2048-token prompts of a 13B-shaped layer, plain causal attention
        _query("query_prompt_13b", S=4, new_lo=2048, new_hi=2048, q_heads=40, heads=40),
        # two long prompts of a grouped-query layer whose scores are capped, queries a view of the projection
        _query("query_prompt_gqa70b_cap", S=2, new_lo=4096, new_hi=4096, q_heads=64, heads=8, cap=50.0, packed=True),
        # chunked prefill: the next 512 tokens of four long documents, FP8 cache
        _query("query_chunk_gqa70b_fp8", pool="fp8", S=4, new_lo=512, new_hi=512, past_lo=15000, past_hi=16000,
               q_heads=64, heads=8),
        # a ragged batch of prompts with a part seen both ways (an image or an instruction), small heads
        _query("query_ragged_prefix", S=24, new_lo=16, new_hi=4096, q_heads=20, heads=5, d=64, B=8, mask="prefix"),
        # packed documents of odd lengths with a distance bias, 4-bit cache
        _query("query_docs_bias_int4", pool="int4", S=3, new_lo=3001, new_hi=3001, q_heads=32, heads=32, mask="docs",
               slopes=True),
        # one decode step of the grouped-query layer, capped scores
        _query("query_decode_gqa70b_cap", S=32, past_lo=4095, past_hi=4095, q_heads=64, heads=8, cap=50.0),
        # one decode step of a small 7B-shaped batch with a distance bias
        _query("query_decode_7b_bias", S=8, past_lo=512, past_hi=2047, slopes=True),
        # checking five drafted tokens per sequence over ragged FP8 contexts
        _query("query_verify_fp8", pool="fp8", S=64, new_lo=5, new_hi=5, past_lo=16, past_hi=16384, q_heads=16,
               heads=8, B=32),
        # one decode step's tokens of a model with three position axes: latency only
        {"name": "rope_axes_decode", "op": "rope", "pool": "f16", "in": "f16", "n": 8, "q_heads": 64, "heads": 8,
         "d": 128, "rot": 128, "sections": "16,24,24", "interleaved": False, "pairs": "half", "B": 16,
         "packed": False, "pad": 0, "prefill": False},
        # a long prompt with images, q, k and v as views of one packed projection
        {"name": "rope_axes_prompt_gqa70b", "op": "rope", "pool": "f16", "in": "f16", "n": 8192, "q_heads": 64,
         "heads": 8, "d": 128, "rot": 128, "sections": "16,24,24", "interleaved": False, "pairs": "half", "B": 16,
         "packed": True, "pad": 0, "prefill": True},
        # an odd prompt with padding, axes in turn over the pairs, float32 projections, FP8 cache
        {"name": "rope_axes_odd_fp8", "op": "rope", "pool": "fp8", "in": "f32", "n": 1001, "q_heads": 10, "heads": 5,
         "d": 64, "rot": 64, "sections": "11,11,10", "interleaved": True, "pairs": "adjacent", "B": 8,
         "packed": False, "pad": 7, "prefill": True},
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    d, B = rng.choice([64, 128, 128]), rng.choice([8, 16, 32])
    if rng.random() < 0.25:
        heads, rot = rng.choice([1, 2, 3, 5, 8, 16, 32, 40]), rng.choice([d, d, d // 2])
        pool, axes = rng.choice(["f16", "fp8", "int4"]), rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, rot // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
        return {"op": "rope", "pool": pool, "in": "f16" if pool == "f16" else rng.choice(["f16", "f32"]),
                "n": _log(rng, 1, 4096), "q_heads": heads * rng.choice([1, 1, 2]), "heads": heads, "d": d, "rot": rot,
                "sections": ",".join(map(str, sections)), "interleaved": rng.random() < 0.4,
                "pairs": rng.choice(["half", "adjacent"]), "B": B, "packed": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 5]), "prefill": rng.random() < 0.5}
    group = rng.choice([1, 1, 2, 4, 8])
    heads = rng.choice([1, 2, 3, 5, 8, 16, 32, 40] if group == 1 else [1, 2, 3, 5, 8] if group < 8 else [1, 2, 3, 5])
    mask = rng.choice(["causal", "causal", "prefix", "docs"])
    more = {"pool": rng.choice(["f16", "f16", "fp8", "int4"]), "q_heads": heads * group, "heads": heads, "d": d, "B": B,
            "mask": mask, "window": rng.choice([0, 0, 100, 1000]) if mask == "causal" else 0,
            "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "slopes": rng.random() < 0.3, "packed": rng.random() < 0.3}
    kind = rng.choice(["prompt", "prompt", "chunk", "step", "step"])
    if kind == "prompt":
        hi, past = _log(rng, 8, 4096), 0
        S = _log(rng, 1, max(1, min(32, 12000 // hi)))
        lo = _log(rng, 1, hi)
    elif kind == "chunk":
        hi, past = _log(rng, 17, 512), _log(rng, 64, 16384)
        S = _log(rng, 1, max(1, min(8, 50_000 // past)))
        lo = _log(rng, 1, hi)
    else:
        hi, past = rng.choice([1, 1, 1, 2, 5, 8]), _log(rng, 16, 32768)
        S = _log(rng, 1, max(1, min(64, 1_000_000 // (past * heads))))
        lo = rng.choice([1, hi])
    c = _query("", S=S, new_lo=lo, new_hi=hi, past_lo=_log(rng, 1, past) if past else 0, past_hi=past, **more)
    del c["name"]
    return c


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


def _tokens(st, which, blk, off):
    """float32 [n, H, d]: K ("k") or V ("v") of tokens (block, offset)."""
    pool, d = st[which + "_pool"], st["case"]["d"]
    kind = st["case"]["pool"]
    if kind == "int4":
        return (_read_k if which == "k" else _read_v)(pool, d, blk, off)
    x = pool[blk, :, off]
    if kind == "fp8":
        return x.view(F8).float() * st[which + "_scale"][blk][:, None, None]
    return x.float()


# ------------------------------------------------------------------------------------ inputs

def _lengths(case):
    """(new tokens, context length) of each sequence: sizes belong to the case, values to the seed."""
    rng = np.random.default_rng([case["S"], case["new_lo"], case["new_hi"], case["past_lo"], case["past_hi"]])

    def some(lo, hi):
        if lo >= hi:
            return np.full(case["S"], hi, dtype=np.int64)
        u = rng.uniform(math.log(lo), math.log(hi + 1), case["S"])
        return np.clip(np.floor(np.exp(u)).astype(np.int64), lo, hi)

    new = some(case["new_lo"], case["new_hi"])
    return new, new + some(case["past_lo"], case["past_hi"])


def _ranges(case):
    """Per new token: position, first and end of the positions it sees (before the window): int64 [n, 3]."""
    rng = np.random.default_rng([case["S"], case["new_hi"], case["past_hi"], 7])
    rows = []
    for n, c in zip(*_lengths(case)):
        p = np.arange(c - n, c)
        lo, hi = np.zeros_like(p), p + 1
        if case["mask"] == "prefix":                 # the past and the first half of the new tokens
            hi = np.maximum(hi, c - n + n // 2)
        elif case["mask"] == "docs":                 # documents of 50 to 1500 tokens, one after the other
            starts, at = [0], int(rng.integers(50, 1501))
            while at < c:
                starts.append(at)
                at += int(rng.integers(50, 1501))
            starts = np.array(starts)
            lo = starts[np.searchsorted(starts, p, side="right") - 1]
        rows.append(np.stack((p, lo, hi), 1))
    return np.concatenate(rows)


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


def _pair_axis(case):
    """The axis of each rotated pair: sections one after the other, or in turn until a section is used up."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["interleaved"]:
        return [a for a, k in enumerate(left) for _ in range(k)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _axis_positions(case, axes, rng):
    """int32 [axes, n]: text (all axes alike) and images (one time, rows and columns of a grid) in turn;
    decode: one token each of sequences at any position."""
    n = case["n"]
    if not case["prefill"]:
        return rng.integers(0, TABLE_LEN, (axes, n)).astype(np.int32)
    pos, at, i = np.zeros((axes, n), dtype=np.int64), int(rng.integers(0, TABLE_LEN - n)), 0
    while i < n:
        k = int(rng.integers(1, 200))
        m = min(k, n - i)
        pos[:, i:i + m] = at + np.arange(m)
        i, at = i + m, at + m
        h, w = (int(x) for x in rng.integers(2, 33, 2))
        m = min(h * w, n - i)
        if m <= 0:
            break
        cell = np.arange(m)
        pos[:, i:i + m] = at
        pos[-2, i:i + m] += cell // w
        pos[-1, i:i + m] += cell % w
        i, at = i + m, at + max(h, w)
    return np.minimum(pos, TABLE_LEN - 1).astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng([int(seed), 1])
    H, Hq, d, B, pool = case["heads"], case["q_heads"], case["d"], case["B"], case["pool"]
    st = {"case": case}

    def pools(nb, fill):
        """K and V tensors: the cache's own with `own`, else plain tensors of the same layout."""
        shape, dt = _pool_shape(pool, nb, H, B, d)
        st["cache"] = None
        if own:
            from paged_kv_cache_169_gb300.cache import PagedKVCache
            st["cache"] = PagedKVCache(1, nb, B, H, d, pool)
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

    if case["op"] == "query":
        new, ctx = _lengths(case)
        n = int(new.sum())
        per = -(-ctx // B)
        nb, width = int(per.sum()) + 3, int(per.max())
        perm = rng.permutation(nb).astype(np.int32)
        tab = np.full((case["S"], width), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(per):
            tab[s, :k] = perm[at:at + k]
            at += k
        pools(nb, True)
        st["new_host"], st["ctx_host"] = new.tolist(), ctx.tolist()
        st["max_queries"], st["max_context"] = int(new.max()), int(ctx.max())
        st["tables"] = torch.from_numpy(tab).cuda()
        st["lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
        st["starts"] = torch.from_numpy(np.concatenate(([0], np.cumsum(new))).astype(np.int32)).cuda()
        # scores of real models with a cap reach tens, where a cap matters; others a few
        x = torch.randn(n, Hq + 2 * H if case["packed"] else Hq, d, generator=gen, device="cuda")
        st["q"] = (x * (4.0 if case["cap"] else 1.0)).half()[:, :Hq]
        st["out"] = torch.zeros(n, Hq, d, dtype=torch.float16, device="cuda")
        st["scale"] = 1.0 / math.sqrt(d)
        st["ranges"] = st["slopes"] = None
        if case["mask"] != "causal":
            st["ranges"] = torch.from_numpy(_ranges(case)[:, 1:].astype(np.int32)).cuda()
        if case["slopes"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, dtype=torch.float64, device="cuda") / Hq).float()
        if own:
            st["workspace"] = st["cache"].query_workspace(case["S"], Hq, st["max_queries"], st["max_context"],
                                                          window=case["window"])
        return st

    n, pad = case["n"], case["pad"]
    nb = -(-n // B) + 5
    perm = rng.permutation(nb)
    tok = np.arange(n)
    # prefill: a sequence's tokens fill whole blocks in order; decode: one token each, anywhere
    slots = perm[tok // B] * B + tok % B if case["prefill"] else rng.permutation(nb * B)[:n]
    if pad:
        slots[pad - 1::pad] = -1
    st["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
    pools(nb, False)
    dt = IN_DTYPE[case["in"]]
    if case["packed"]:
        x = torch.randn(n, Hq + 2 * H, d, generator=gen, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        st["q"], st["k"], st["v"] = (torch.randn(n, h, d, generator=gen, device="cuda").to(dt) for h in (Hq, H, H))
    axis = _pair_axis(case)
    st["axis"] = torch.tensor(axis, device="cuda")
    st["positions"] = torch.from_numpy(_axis_positions(case, max(axis) + 1, rng)).cuda()
    # the rotation table a program keeps: cosines then sines of each position's angles
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
    ang = torch.arange(TABLE_LEN, dtype=torch.float64, device="cuda")[:, None] * freq
    st["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float().contiguous()
    st["q_out"] = torch.zeros(n, Hq, d, dtype=torch.float16, device="cuda")
    if pool == "int4":
        st["k_back"], st["v_back"] = (torch.zeros(n, H, d, dtype=torch.float16, device="cuda") for _ in range(2))
    if own:
        from paged_kv_cache_169_gb300.cache import rope_axes
        st["rope_axes"] = rope_axes(axis)
    return st


# ------------------------------------------------------------------------------------ one pass

def _plain_query(st):
    case = st["case"]
    H, B, cap = case["heads"], case["B"], case["cap"]
    G = case["q_heads"] // H
    at = 0
    for s, (n, c) in enumerate(zip(st["new_host"], st["ctx_host"])):
        rows = slice(at, at + n)
        at += n
        j = torch.arange(c, device="cuda")
        blk, off = st["tables"][s].long()[j // B], j % B
        k, v = (_tokens(st, w, blk, off).transpose(0, 1) for w in "kv")               # [H, c, d]
        p = torch.arange(c - n, c, device="cuda")
        first, last = torch.zeros_like(p), p + 1
        if st["ranges"] is not None:
            first, last = st["ranges"][rows].long().unbind(1)
        if case["window"]:
            first = torch.maximum(first, p - case["window"] + 1)
        seen = (j >= first[:, None]) & (j < last[:, None])
        far = (p[:, None] - j).abs().float()
        q = st["q"][rows].float()
        step = max(1, (1 << 30) // (n * c * G))                                       # K/V heads at a time
        for h in range(0, H, step):
            m = min(step, H - h)
            x = torch.matmul(q[:, h * G:(h + m) * G].transpose(0, 1).reshape(m, G * n, -1),
                             k[h:h + m].transpose(1, 2)).view(m, G, n, c).mul_(st["scale"])
            if cap:
                x = x.div_(cap).tanh_().mul_(cap)
            if st["slopes"] is not None:
                x = x - st["slopes"][h * G:(h + m) * G].view(m, G, 1, 1) * far
            x = x.masked_fill_(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
            total = x.sum(-1, keepdim=True)
            o = torch.matmul(x.view(m, G * n, c), v[h:h + m]).view(m, G, n, -1)
            o = torch.where(total > 0, o / total, 0.0)
            st["out"][rows, h * G:(h + m) * G] = o.flatten(0, 1).transpose(0, 1).half()
    return {"out": st["out"]}


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
    at = st["positions"].long()[st["axis"]].T                       # [n, rot/2]: each pair's position
    pair = torch.arange(rot // 2, device="cuda")
    cos, sin = st["cos_sin"][at, pair], st["cos_sin"][at, rot // 2 + pair]
    q = _rotate(st["q"].float(), cos, sin, rot, case["pairs"])
    st["q_out"].copy_(torch.where(live[:, None, None], q.half(), st["q_out"]))
    # a padding token stands for the first live one: the same values at the same place again
    src = torch.where(live, torch.arange(case["n"], device=live.device), live.int().argmax())
    blk, off = st["slots"][src] // B, st["slots"][src] % B
    k = _rotate(st["k"].float(), cos, sin, rot, case["pairs"])[src]
    v = st["v"].float()[src]
    if pool == "int4":
        _write(st["k_pool"], st["v_pool"], k, v, d, blk, off)
        at = st["slots"].clamp(min=0)
        for w in "kv":
            x = _tokens(st, w, at // B, at % B)
            st[w + "_back"].copy_(torch.where(live[:, None, None], x.half(), st[w + "_back"]))
        return {"q": st["q_out"], "k": st["k_back"], "v": st["v_back"]}
    for w, x in (("k", k), ("v", v)):
        if pool == "fp8":
            x = (x / st[w + "_scale"][blk][:, None, None]).clamp(-448, 448).to(F8).view(torch.uint8)
        st[w + "_pool"][blk, :, off] = x if pool == "fp8" else x.half()
    return _pools_out(st)


def _pools_out(st):
    f8 = st["case"]["pool"] == "fp8"
    return {"q": st["q_out"], "k": st["k_pool"].view(F8) if f8 else st["k_pool"],
            "v": st["v_pool"].view(F8) if f8 else st["v_pool"]}


def _own(st):
    from paged_kv_cache_169_gb300 import abi
    case, cache = st["case"], st["cache"]
    if case["op"] == "query":
        return {"out": cache.query_attention(
            0, st["q"], st["starts"], st["tables"], st["lens"], st["max_queries"], st["max_context"], st["scale"],
            window=case["window"], score_cap=case["cap"], slopes=st["slopes"], ranges=st["ranges"], out=st["out"],
            workspace=st["workspace"], flags=abi.KV_DECODE_WORKSPACE_ZEROED | abi.KV_DECODE_PDL)}
    cache.append_rope_axes(0, st["k"], st["v"], st["slots"], st["positions"], st["rope_axes"], st["cos_sin"],
                           q=st["q"], q_out=st["q_out"], adjacent_pairs=case["pairs"] == "adjacent")
    if case["pool"] == "int4":
        k, v = cache.gather(0, st["slots"], k_out=st["k_back"], v_out=st["v_back"])
        return {"q": st["q_out"], "k": k, "v": v}
    return _pools_out(st)


def run(state):
    if own:
        return _own(state)
    return {"query": _plain_query, "rope": _plain_rope}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ work

def _row_bytes(pool, d):
    """Bytes of one token of one head in a pool."""
    return {"f16": 2 * d, "fp8": d, "int4": d // 2 + d // 16}[pool]


def work(case):
    H, Hq, d = case["heads"], case["q_heads"], case["d"]
    if case["op"] == "query":
        new, ctx = _lengths(case)
        n, at, read, pairs = int(new.sum()), 0, 0, 0
        rows = _ranges(case)
        first = np.maximum(rows[:, 1], rows[:, 0] - case["window"] + 1) if case["window"] else rows[:, 1]
        for k, c in zip(new, ctx):
            lo, hi = first[at:at + k], np.minimum(rows[at:at + k, 2], c)
            at += k
            pairs += int((hi - lo).sum())
            read += int(hi.max() - lo.min())
        extra = 8 * n if case["mask"] != "causal" else 0
        return {"bytes": 4 * n * Hq * d + 2 * read * H * _row_bytes(case["pool"], d) + 4 * read // case["B"] + extra,
                "flops": 4 * pairs * Hq * d}
    n = case["n"] - (case["n"] // case["pad"] if case["pad"] else 0)
    i = {"f16": 2, "f32": 4}[case["in"]]
    axes = case["sections"].count(",") + 1
    back = 2 * n * H * (_row_bytes("int4", d) + 2 * d) if case["pool"] == "int4" else 0
    return {"bytes": n * (Hq * d * (i + 2) + 2 * H * (i * d + _row_bytes(case["pool"], d))) +
            (8 + 4 * axes) * case["n"] + 4 * case["rot"] * n + back,
            "flops": 3 * n * (Hq + H) * case["rot"] + 3 * n * 2 * H * d}


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
    if case["op"] == "rope":
        slots, rot, out = st["slots"], case["rot"], {}
        live = torch.nonzero(slots >= 0)[:, 0]
        blk, off = slots[live] // B, slots[live] % B
        pair = torch.arange(rot // 2, device="cuda")
        z = torch.empty(case["n"], rot // 2, dtype=torch.complex128, device="cuda")
        for i, a in enumerate(_pair_axis(case)):
            row = st["cos_sin"][st["positions"][a].long()].double()
            z[:, i] = torch.complex(row[:, i], row[:, rot // 2 + i])
        a, b = (pair, pair + rot // 2) if case["pairs"] == "half" else (2 * pair, 2 * pair + 1)
        for w in "qkv":
            x = st[w].double()
            if w != "v":
                y = torch.complex(x[..., a], x[..., b]) * z[:, None]
                x = x.index_copy(2, a, y.real).index_copy(2, b, y.imag)
            x = x[live]
            if w == "q" or case["pool"] == "int4":
                x = x if w == "q" else _nearest4(x)
                out[w] = torch.zeros(case["n"], *x.shape[1:], dtype=torch.float64, device="cuda").index_copy_(0, live, x)
                continue
            if case["pool"] == "fp8":
                x = (x / st[w + "_scale"].double()[blk][:, None, None]).clamp(-448, 448)
            out[w] = torch.zeros(st[w + "_pool"].shape, dtype=torch.float64, device="cuda")
            out[w][blk, :, off] = x
        return out
    if work(case)["flops"] > 4e12:
        return None
    G = case["q_heads"] // H
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    rows = torch.from_numpy(_ranges(case)).cuda()
    end = torch.tensor(st["new_host"]).cumsum(0).tolist()
    for s, (n, c, e) in enumerate(zip(st["new_host"], st["ctx_host"], end)):
        pos, first, last = rows[e - n:e].T[..., None]
        key = torch.arange(c, device="cuda")[None]
        hidden = (key < first) | (key >= last)
        if case["window"]:
            hidden |= pos - key >= case["window"]
        blk, off = st["tables"][s].long()[key[0] // B], key[0] % B
        for h in range(H):
            kv = []
            for w in "kv":
                pool = st[w + "_pool"][:, h:h + 1]
                if case["pool"] == "int4":
                    x = _token_values(pool, w, d, blk, off)
                elif case["pool"] == "fp8":
                    x = pool.view(F8)[blk, :, off].double() * st[w + "_scale"].double()[blk][:, None, None]
                else:
                    x = pool[blk, :, off].double()
                kv.append(x[:, 0])
            for g in range(h * G, (h + 1) * G):
                x = torch.mm(st["q"][e - n:e, g].double(), kv[0].T) * st["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["slopes"]:
                    x = x - st["slopes"][g].double() * (pos - key).abs()
                w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[e - n:e, g] = torch.mm(w.nan_to_num(0.0), kv[1])
    return {"out": out}
