"""GPU: kv_gather over slots in every order that its kernels tell apart, and the calls of a prompt in a row."""

import numpy as np
import pytest
import torch

from oracle import int4 as O4
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_table

pytestmark = pytest.mark.gpu

NP = {"f16": np.float16, "f32": np.float32}


def slots_of(order, rng, n, nb, B):
    perm = rng.permutation(nb)
    i = np.arange(n)
    if order == "aligned":                             # a cached prefix from its first token on
        s = perm[i // B] * B + i % B
    elif order == "mid_oct":                           # from its sixth on
        s = perm[(i + 5) // B] * B + (i + 5) % B
    elif order == "padded":                            # a padding row inside an oct, another at the end of one
        s = perm[i // B] * B + i % B
        s[11::40] = -1
        s[23::64] = -7
    elif order == "odd_lengths":                       # several prefixes, each from a block's start
        s, at = [], 0
        while len(s) < n:
            m = int(rng.integers(1, 3 * B))
            blocks = rng.integers(0, nb, -(-m // B))
            s += [blocks[j // B] * B + j % B for j in range(m)]
        s = np.array(s[:n])
    else:                                              # octs whose tokens come in another order
        s = perm[i // B] * B + i % B
        s[8:16] = s[8:16][::-1]
        s[24:26] = s[[25, 24]]
    return s.astype(np.int64)


@pytest.mark.parametrize("order", ["aligned", "mid_oct", "padded", "odd_lengths", "turned"])
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("n,H,d,B", [(8, 1, 64, 8), (125, 3, 128, 16), (131, 9, 64, 32), (600, 2, 128, 8), (77, 40, 64, 16)])
def test_int4_gather_orders(order, out, n, H, d, B):
    if order == "turned" and n < 26:
        n = 26
    rng = np.random.default_rng(n + H)
    nb = -(-(n + 5) // B) + 2
    cache = PagedKVCache(1, nb, B, H, d, "int4")
    pools = []
    for t in (cache.k[0], cache.v[0]):
        a = rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)
        a[..., 4 * d:] %= 199                          # any finite scale
        t.copy_(torch.from_numpy(a))
        pools.append(a)
    slots = slots_of(order, rng, n, nb, B)
    dt = torch.float16 if out == "f16" else torch.float32
    got = [torch.full((n, H, d), 2.5, dtype=dt, device="cuda") for _ in range(2)]
    cache.gather(0, torch.from_numpy(slots).cuda(), k_out=got[0], v_out=got[1])
    assert cache.device_error() == 0
    live = slots >= 0
    for which, g, a in zip("kv", got, pools):
        want = np.full((n, H, d), 2.5, dtype=NP[out])
        want[live] = O4.token_values(a, which, d, slots[live] // B, slots[live] % B)
        assert np.array_equal(g.cpu().numpy(), want), which
    cache.close()


@pytest.mark.parametrize("pool", ["f16", "int4"])
@pytest.mark.parametrize("G", [1, 8])
def test_rotated_append_then_attention_under_programmatic_launch(pool, G):
    """A layer's two launches with KV_DECODE_PDL, captured and replayed on new inputs: the bits of calls
    one after the other."""
    B, H, d, S, ctx = 16, 2, 128, 5, 90
    caches = [PagedKVCache(1, 40, B, H, d, pool) for _ in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(G)
    old = [torch.randn(40 * B, H, d, generator=gen, device="cuda").half() for _ in range(2)]
    for c in caches:
        c.append(0, *old, torch.arange(40 * B, device="cuda"))
    tab = torch.randperm(40, generator=gen, device="cuda")[:S * 6].to(torch.int32).reshape(S, 6)
    lens = torch.tensor([ctx, 1, 33, 64, 17], dtype=torch.int32, device="cuda")
    pos = lens - 1
    slots = tab.gather(1, (pos // B).long()[:, None])[:, 0].long() * B + pos % B
    table = rope_table(128, d)
    q = torch.randn(S, H * G, d, generator=gen, device="cuda").half()
    k, v = (torch.randn(S, H, d, generator=gen, device="cuda").half() for _ in range(2))
    qr = [torch.zeros_like(q) for _ in range(2)]
    out = [torch.zeros(S, H * G, d, device="cuda") for _ in range(2)]
    ws = [caches[0].zeroed_workspace(S, ctx, num_q_heads=H * G) for _ in range(2)]

    def step(i, flags, stream=None):
        caches[i].append_rope(0, k, v, slots, pos, table, q=q, q_out=qr[i], flags=flags, stream=stream)
        more = abi.KV_DECODE_WORKSPACE_ZEROED | (flags and flags | abi.KV_DECODE_EARLY_TABLES)
        caches[i].attention_ex(0, qr[i], tab, lens, ctx, 0.1, out=out[i], workspace=ws[i], flags=more, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            step(0, abi.KV_DECODE_PDL, side)
    torch.cuda.synchronize()
    for turn in range(3):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        step(1, 0)
        assert torch.equal(qr[0], qr[1]) and torch.equal(out[0], out[1]), turn
        assert torch.equal(caches[0].k[0], caches[1].k[0]) and torch.equal(caches[0].v[0], caches[1].v[0])
    for c in caches:
        assert c.device_error() == 0
        c.close()
