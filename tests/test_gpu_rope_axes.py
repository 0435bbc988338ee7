"""GPU: kv_append_rope_axes.  Each pair turns by its own axis' position: the same float32 roundings as
kv_append_rope over a table whose row for a token is put together pair by pair, so the results are compared
bit for bit with that call and, through it, with the oracle."""

import numpy as np
import pytest
import torch

from oracle import rope as OR
from paged_kv_cache_169_gb300 import abi
from paged_kv_cache_169_gb300.cache import PagedKVCache, rope_axes, rope_table

pytestmark = pytest.mark.gpu


def layout(kind, pairs, axes, rng):
    if kind == "sections":
        cuts = np.sort(rng.choice(np.arange(1, pairs), axes - 1, replace=False))
        return np.searchsorted(cuts, np.arange(pairs), side="right")
    if kind == "turns":
        return np.arange(pairs) % axes
    a = rng.integers(0, axes, pairs)
    a[0] = axes - 1
    return a


def case(pool, in_dtype, d, rot, adjacent, B, n, axes, kind, H=3, Hq=5, packed=False, pad=(), in_place=False, seed=0):
    rng = np.random.default_rng(seed)
    nb, T = -(-n // B) + 3, 90
    ax = layout(kind, rot // 2, axes, rng)
    pos = rng.integers(0, T, (axes, n)).astype(np.int32)
    slots = rng.permutation(nb * B)[:n].astype(np.int64)
    for i in pad:
        slots[i], pos[:, i] = -2, -9
    tab = rng.standard_normal((T, rot)).astype(np.float32)
    live = slots >= 0
    # each token's row: pair i from the row of its axis' position
    at = np.where(live, pos, 0)[ax]                                    # [rot/2, n]
    rows = np.concatenate((tab[at, np.arange(rot // 2)[:, None]].T,
                           tab[at, rot // 2 + np.arange(rot // 2)[:, None]].T), 1)
    rows = np.ascontiguousarray(rows)
    dt = np.float16 if in_dtype == "f16" else np.float32
    q, k, v = (rng.standard_normal((n, h, d)).astype(dt) for h in (Hq, H, H))
    res = []
    for several in (True, False):
        cache = PagedKVCache(1, nb, B, H, d, pool)
        for t in cache.k + cache.v:
            t.view(torch.uint8).zero_()
        if pool == "fp8":
            for t in (cache.k_scale[0], cache.v_scale[0]):
                t.copy_(torch.linspace(0.004, 0.02, t.numel(), device="cuda"))
        if packed:
            x = torch.from_numpy(np.concatenate([q, k, v], 1)).cuda()
            tq, tk, tv = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        else:
            tq, tk, tv = (torch.from_numpy(a).cuda() for a in (q, k, v))
        out = tq if in_place else torch.full((n, Hq, d), 9.5, dtype=torch.float32 if pool == "f32" else torch.float16,
                                             device="cuda")
        ts = torch.from_numpy(slots).cuda()
        if several:
            cache.append_rope_axes(0, tk, tv, ts, torch.from_numpy(pos).cuda(), rope_axes(ax), torch.from_numpy(tab).cuda(),
                                   q=tq, q_out=out, adjacent_pairs=adjacent)
        else:
            one = torch.arange(n, dtype=torch.int32, device="cuda")
            cache.append_rope(0, tk, tv, ts, one, torch.from_numpy(rows).cuda(), q=tq, q_out=out, adjacent_pairs=adjacent)
        assert cache.device_error() == 0
        res.append([out.cpu().numpy()] + [t.cpu().view(torch.uint8).numpy() for t in (cache.k[0], cache.v[0])])
        cache.close()
    for a, b in zip(*res):
        assert np.array_equal(a, b)
    want = OR.rotate(q, rows, rot, adjacent, np.float32).astype(res[0][0].dtype)
    assert np.array_equal(res[0][0][live], want[live])
    if not in_place:
        assert (res[0][0][~live] == 9.5).all()


@pytest.mark.parametrize("pool,in_dtype", [("f32", "f32"), ("f16", "f16"), ("fp8", "f16"), ("fp8", "f32"),
                                           ("int4", "f16"), ("int4", "f32")])
@pytest.mark.parametrize("d,rot,adjacent,B,axes,kind", [(128, 128, False, 16, 3, "sections"), (128, 64, True, 8, 3, "turns"),
                                                        (128, 96, False, 32, 4, "any"), (64, 64, False, 16, 2, "turns"),
                                                        (64, 16, True, 32, 4, "any"), (64, 48, True, 8, 2, "sections"),
                                                        (64, 32, False, 8, 3, "any"), (128, 16, False, 16, 1, "any")])
def test_every_pool(pool, in_dtype, d, rot, adjacent, B, axes, kind):
    case(pool, in_dtype, d, rot, adjacent, B, 13, axes, kind, pad=(4, 11), seed=d + rot + B)


@pytest.mark.parametrize("n", [1, 2, 3, 64, 701])
@pytest.mark.parametrize("pool", ["f16", "int4"])
def test_lengths(n, pool):
    case(pool, "f16", 128, 128, False, 16, n, 3, "sections", H=1, Hq=4, packed=True, seed=n)
    case(pool, "f16", 64, 32, True, 8, n, 2, "any", H=5, Hq=1, seed=n, pad=(n - 1,) if n > 1 else ())
    case(pool, "f16", 64, 64, False, 8, n, 4, "turns", H=2, Hq=2, seed=n, in_place=True)


def test_bad_position_on_any_axis_skips_the_token():
    cache = PagedKVCache(1, 4, 16, 2, 64, "f16")
    for t in (cache.k[0], cache.v[0]):
        t.fill_(3.0)
    k = torch.randn(4, 2, 64, device="cuda").half()
    tab, ax = rope_table(10, 64), rope_axes([0, 1, 2, 0] * 8)
    slots = torch.arange(4, device="cuda")
    for axis in range(3):
        for bad in (-1, 10, 2 ** 31 - 1, -2 ** 31):
            pos = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
            pos[axis, 2] = bad
            cache.append_rope_axes(0, k, k, slots, pos, ax, tab)
            assert cache.device_error() == abi.KV_DEVERR_POSITION
            assert torch.equal(cache.k[0][0][:, [0, 1, 3]].transpose(0, 1), k[[0, 1, 3]])
            assert (cache.k[0][0][:, 2] == 3).all() and (cache.v[0][0][:, 2] == 3).all()
    for bad in (dict(positions=pos[:2]), dict(positions=pos[0]), dict(positions=pos[:, :3]), dict(axes=rope_axes([0, 1, 2, 0])),
                dict(positions=pos.long()), dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            cache.append_rope_axes(**{**dict(layer=0, k=k, v=k, slot_mapping=slots, positions=pos, axes=ax, cos_sin=tab), **bad})
    cache.append_rope_axes(0, k[:0], k[:0], slots[:0], pos[:, :0].contiguous(), ax, tab)
    assert cache.device_error() == 0
    cache.close()
