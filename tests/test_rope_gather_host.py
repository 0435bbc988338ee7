"""Refusals of kv_append_rope, kv_gather, kv_rope_table and of 4-bit pools that need no GPU.

Argument checks read only the pool's descriptor, the first field behind the handle, so a zeroed
buffer that starts with a descriptor stands for a pool: every call here must be refused with
KV_ERR_INVALID_ARG before anything touches a device (the accepted one then fails because the
process has no device, or the buffer's device is not current)."""

import ctypes as C

import pytest

from paged_kv_cache_169_gb300 import abi, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


class _Handle(C.Structure):
    _fields_ = [("desc", abi.kv_pool_desc), ("device", C.c_int), ("rest", C.c_char * 512)]


def pool(dtype=abi.KV_F16, d=128, H=4, B=16):
    h = _Handle()
    h.desc = abi.kv_pool_desc(2, 10, B, H, d, dtype)
    h.device = -7                                          # never the current device
    return h


A = 1 << 20                                                # an aligned address nobody reads


def rope_args(**kw):
    a = abi.kv_rope_args()
    base = dict(layer=1, q=A, num_q_heads=8, q_out=2 * A, k=3 * A, v=4 * A, in_dtype=abi.KV_F16, q_stride=1024,
                k_stride=512, v_stride=512, q_out_stride=1024, slot_mapping=5 * A, positions=6 * A, cos_sin=7 * A,
                table_len=100, rot_dim=128, adjacent_pairs=0, num_tokens=3, flags=0)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def status(fn, *args):
    try:
        fn(*args)
    except abi.KvError as e:
        return e.status
    return 0


BAD_ROPE = [dict(layer=2), dict(layer=-1), dict(num_tokens=-1), dict(k=None), dict(v=None), dict(slot_mapping=None),
            dict(positions=None), dict(cos_sin=None), dict(k=3 * A + 8), dict(v=4 * A + 2), dict(q=A + 8),
            dict(q_out=2 * A + 8), dict(q_out=None), dict(cos_sin=7 * A + 4), dict(rot_dim=0), dict(rot_dim=8),
            dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=-16), dict(table_len=0), dict(adjacent_pairs=2),
            dict(in_dtype=abi.KV_F32), dict(in_dtype=abi.KV_INT4), dict(k_stride=504), dict(v_stride=0),
            dict(q_stride=1023), dict(q_out_stride=512), dict(k_stride=516), dict(k_stride=1 << 28),
            dict(k_stride=-512), dict(num_q_heads=0), dict(num_q_heads=2049), dict(flags=1), dict(flags=64),
            dict(q_out=A, q_out_stride=2048)]


@pytest.mark.parametrize("bad", BAD_ROPE, ids=str)
def test_append_rope_refuses(bad):
    h = pool()
    assert status(abi.kv_append_rope, C.addressof(h), rope_args(**bad)) == abi.KV_ERR_INVALID_ARG


def test_append_rope_edges():
    h = pool()
    assert status(abi.kv_append_rope, 0, rope_args()) == abi.KV_ERR_INVALID_ARG
    assert status(abi.kv_append_rope, C.addressof(h), rope_args(num_tokens=0, k=None)) == 0
    # a float32 projection into a pool that keeps float16, in place: the rows would overlap
    h8 = pool(abi.KV_INT4)
    assert status(abi.kv_append_rope, C.addressof(h8),
                  rope_args(in_dtype=abi.KV_F32, q_out=A)) == abi.KV_ERR_INVALID_ARG
    # every argument right, but another device than the pool's
    assert status(abi.kv_append_rope, C.addressof(h), rope_args()) == abi.KV_ERR_INVALID_ARG


def test_gather_refuses():
    h, f32 = pool(abi.KV_INT4), pool(abi.KV_F32)
    ok = (C.addressof(h), 0, A, 3, 2 * A, 3 * A, abi.KV_F16)

    def call(**kw):
        names = ("pool", "layer", "slots", "n", "k", "v", "dt")
        return status(abi.kv_gather, *[kw.get(n, v) for n, v in zip(names, ok)])

    for bad in (dict(pool=0), dict(layer=2), dict(layer=-1), dict(n=-1), dict(slots=0), dict(k=0), dict(v=0),
                dict(k=2 * A + 8), dict(v=3 * A + 4), dict(dt=abi.KV_INT4), dict(dt=abi.KV_FP8_E4M3), dict(dt=9),
                dict(pool=C.addressof(f32))):
        assert call(**bad) == abi.KV_ERR_INVALID_ARG, bad
    assert call(n=0, k=0) == 0


def test_rope_table_refuses():
    for bad in ((0, 10, 64, 1e4, 1.0), (A + 4, 10, 64, 1e4, 1.0), (A, 0, 64, 1e4, 1.0), (A, (1 << 24) + 1, 64, 1e4, 1.0),
                (A, 10, 40, 1e4, 1.0), (A, 10, 272, 1e4, 1.0), (A, 10, 64, 1.0, 1.0), (A, 10, 64, float("nan"), 1.0),
                (A, 10, 64, float("inf"), 1.0), (A, 10, 64, 1e4, 0.0), (A, 10, 64, 1e4, float("inf"))):
        assert status(abi.kv_rope_table, *bad) == abi.KV_ERR_INVALID_ARG, bad


def test_int4_pool_takes_no_scales_and_no_prefix_groups():
    with pytest.raises(abi.KvError) as e:
        abi.kv_pool_create(1, 4, 16, 2, 64, abi.KV_INT4, [256], [256], [512], [512])
    assert e.value.status == abi.KV_ERR_INVALID_ARG
    h = pool(abi.KV_INT4)
    assert abi.load().kv_swap_bytes(C.addressof(h), 3, 0, 2) == 3 * 2 * 2 * 4 * 16 * (64 + 8)
    a = abi.kv_decode_args()
    a.q, a.out, a.block_tables, a.context_lens, a.workspace = A, A, A, A, A
    a.max_blocks_per_seq, a.batch, a.max_context, a.scale, a.workspace_bytes = 4, 2, 64, 1.0, 1 << 30
    a.prefix_groups, a.num_prefix_groups = A, 1
    assert status(abi.paged_decode_attention_ex, C.addressof(h), a) == abi.KV_ERR_UNSUPPORTED


def test_rope_args_layout_matches_header(tmp_path, monkeypatch):
    """The binding's kv_rope_args has the C header's layout (the check of test_abi_layout)."""
    import json
    import os
    import shutil
    import subprocess

    import test_abi_layout as L
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no host C compiler")
    monkeypatch.setattr(L, "STRUCTS", {"kv_rope_args": abi.kv_rope_args})
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(L._probe_source())
    subprocess.run([cc, "-std=c99", "-I", os.path.join(L.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    want = json.loads(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout)["kv_rope_args"]
    assert C.sizeof(abi.kv_rope_args) == want["size"]
    for field, _ in abi.kv_rope_args._fields_:
        assert getattr(abi.kv_rope_args, field).offset == want[field], field
