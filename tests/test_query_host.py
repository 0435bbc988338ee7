"""Refusals of paged_query_attention, its workspace size and kv_append_rope_axes that need no GPU (a zeroed
buffer that starts with a descriptor stands for a pool), and the binding's layouts."""

import ctypes as C
import json
import os
import shutil
import subprocess

import pytest

import test_abi_layout as L
import test_rope_gather_host as R
from paged_kv_cache_169_gb300 import abi, build
from paged_kv_cache_169_gb300.cache import rope_axes

A = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load()


def query_args(**kw):
    a = abi.kv_query_args()
    base = dict(layer=1, q=A, num_q_heads=8, q_stride=1024, out=2 * A, out_stride=1024, query_start=3 * A, num_tokens=30,
                max_queries=20, block_tables=4 * A, max_blocks_per_seq=5, context_lens=5 * A, batch=3, max_context=80,
                window=0, scale=0.1, score_cap=0.0, workspace=6 * A, workspace_bytes=1 << 40, flags=0)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


NAN, INF = float("nan"), float("inf")
BAD = [dict(layer=2), dict(layer=-1), dict(batch=-1), dict(batch=65537), dict(num_tokens=-1),
       dict(num_tokens=(1 << 24) + 1), dict(max_queries=-1), dict(max_queries=31), dict(max_context=-1),
       dict(max_context=(1 << 24) + 1), dict(window=-1), dict(num_q_heads=0), dict(num_q_heads=6), dict(num_q_heads=12),
       dict(num_q_heads=64), dict(num_q_heads=-4), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF),
       dict(score_cap=-1.0), dict(score_cap=NAN), dict(score_cap=INF), dict(flags=4), dict(flags=8), dict(flags=64),
       dict(q=None), dict(out=None), dict(query_start=None), dict(block_tables=None), dict(context_lens=None),
       dict(workspace=None), dict(max_blocks_per_seq=0), dict(q=A + 8), dict(out=2 * A + 2), dict(workspace=6 * A + 128),
       dict(ranges=7 * A + 4), dict(slopes=7 * A + 2), dict(q_stride=1023), dict(q_stride=1020), dict(q_stride=512),
       dict(out_stride=0), dict(out_stride=1 << 28), dict(workspace_bytes=0), dict(out=A)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_query_attention_refuses(bad):
    h = R.pool()
    assert R.status(abi.paged_query_attention, C.addressof(h), query_args(**bad)) == abi.KV_ERR_INVALID_ARG


def test_query_attention_edges():
    h = R.pool()
    assert R.status(abi.paged_query_attention, 0, query_args()) == abi.KV_ERR_INVALID_ARG
    assert R.status(abi.paged_query_attention, C.addressof(h), query_args(batch=0, q=None)) == 0
    assert R.status(abi.paged_query_attention, C.addressof(h), query_args(max_queries=0, num_tokens=0, q=None)) == 0
    # every argument right, but another device than the pool's
    for dt in (abi.KV_F32, abi.KV_F16, abi.KV_FP8_E4M3, abi.KV_INT4):
        h = R.pool(dt)
        assert R.status(abi.paged_query_attention, C.addressof(h), query_args()) == abi.KV_ERR_INVALID_ARG


def test_query_workspace_size():
    h = R.pool()
    C.memmove(C.addressof(h) + abi.C.sizeof(abi.kv_pool_desc) + 4, C.byref(C.c_int(152)), 4)    # num_sms
    size = abi.load().paged_query_workspace_size
    assert size(C.addressof(h), C.byref(query_args())) >= 256
    assert size(None, C.byref(query_args())) == 0 and size(C.addressof(h), None) == 0
    for bad in (dict(batch=-1), dict(max_queries=31), dict(num_q_heads=7), dict(window=-2), dict(max_context=-5)):
        assert size(C.addressof(h), C.byref(query_args(**bad))) == 0, bad
    # neither the number of rows nor what the call reads changes the layout
    assert size(C.addressof(h), C.byref(query_args(num_tokens=60, q=None))) == size(C.addressof(h), C.byref(query_args()))


def axes(num=3, stride=3, pairs=None):
    x = abi.kv_rope_axes(num, stride)
    x.pair_axis[:64] = pairs if pairs is not None else [i % num for i in range(64)]
    return x


def call_axes(x, **kw):
    h = R.pool()
    return R.status(abi.kv_append_rope_axes, C.addressof(h), R.rope_args(**kw), x)


@pytest.mark.parametrize("bad", R.BAD_ROPE, ids=str)
def test_append_rope_axes_refuses_what_append_rope_refuses(bad):
    assert call_axes(axes(stride=1000), **bad) == abi.KV_ERR_INVALID_ARG


def test_append_rope_axes_refuses():
    for x in (axes(0, 3, [0] * 64), axes(-1, 3, [0] * 64), axes(5, 3, [0] * 64), axes(stride=2), axes(stride=1 << 31),
              axes(stride=-3), axes(2, 3, [0] * 63 + [2]), axes(1, 3, [255] + [0] * 63)):
        assert call_axes(x) == abi.KV_ERR_INVALID_ARG
    assert call_axes(axes(2, 3, [0] * 63 + [2]), num_tokens=0) == abi.KV_ERR_INVALID_ARG
    assert call_axes(axes(), num_tokens=0, k=None) == 0
    # pairs beyond rot_dim / 2 are not looked at (refused here for the device only)
    assert abi.load().kv_append_rope_axes(C.addressof(R.pool()), C.byref(R.rope_args()), None) == abi.KV_ERR_INVALID_ARG


def test_rope_axes_helper():
    x = rope_axes([0, 1, 2, 2])
    assert x.num_axes == 3 and list(x.pair_axis[:4]) == [0, 1, 2, 2]
    for bad in ([], [4], [-1], [0] * 65):
        with pytest.raises(ValueError):
            rope_axes(bad)


def test_layouts_match_header(tmp_path, monkeypatch):
    """kv_query_args and kv_rope_axes as in the C header (the check of test_abi_layout)."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no host C compiler")
    structs = {"kv_query_args": abi.kv_query_args, "kv_rope_axes": abi.kv_rope_axes}
    monkeypatch.setattr(L, "STRUCTS", structs)
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(L._probe_source())
    subprocess.run([cc, "-std=c99", "-I", os.path.join(L.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = json.loads(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout)
    for name, cls in structs.items():
        assert C.sizeof(cls) == got[name]["size"]
        for field, *_ in cls._fields_:
            assert getattr(cls, field).offset == got[name][field], (name, field)
