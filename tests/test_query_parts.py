"""How paged_query_attention lays out the partial sums of keys cut into parts (csrc/query_parts.h): every place that a
call's rows take lies within the workspace that was asked for, whatever num_tokens, batch and max_queries are."""

import ctypes as C
import os
import shutil
import subprocess

import pytest

import test_query_host as H
import test_rope_gather_host as R
from paged_kv_cache_169_gb300 import abi, build

SMS = 152
SOURCE = """
#include <algorithm>
#include "query_parts.h"
extern "C" void last_place(int sms, int batch, int heads, int group, int tokens, int queries, int context, int window,
                           int64_t* out) {
    const kvp::QueryParts p = kvp::query_parts(sms, batch, heads, group, tokens, queries, context, window);
    // the farthest row: of the last sequence its last, which lies before num_tokens and is one of max_queries
    const int n = std::min(queries, tokens);
    const int64_t row = kvp::part_row(p.by_sequence, queries, batch - 1, tokens - n, n - 1);
    out[0] = p.splits;
    out[1] = p.splits > 1 ? ((p.splits - 1) * p.rows + row) * heads * group + heads * group - 1 : -1;
    out[2] = p.space;
    out[3] = p.rows > row;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host C++ compiler")
    at = tmp_path_factory.mktemp("parts")
    (at / "parts.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(at / "parts.cpp"), "-o",
                    str(at / "parts.so")], check=True)
    return C.CDLL(os.fspath(at / "parts.so"))


def pool(dtype, d, H):
    h = R.pool(dtype, d, H)
    C.memmove(C.addressof(h) + C.sizeof(abi.kv_pool_desc) + 4, C.byref(C.c_int(SMS)), 4)        # num_sms
    return h


@pytest.mark.parametrize("heads,group,d", [(1, 1, 64), (4, 4, 128), (8, 8, 128), (40, 1, 128), (5, 2, 64)])
def test_parts_lie_in_the_workspace(lib, heads, group, d):
    """num_tokens up to far above batch * max_queries: q is a padded buffer."""
    h = pool(abi.KV_F16, d, heads)
    size = abi.load().paged_query_workspace_size
    counters = -(-SMS * 16 // 256) * 256
    out, cut = (C.c_int64 * 4)(), 0
    for batch in (1, 2, 7, 33):
        for queries in (17, 32, 83, 100, 257, 1000):
            for extra in (1, 2, 5, 64, 4096):
                for tokens in (batch * queries * extra, batch * queries * extra + 5, queries, queries + 1):
                    for context in (600, 1024, 5000, 16384, 1 << 20):
                        for window in (0, 700):
                            if queries * group <= 16 or tokens < queries or tokens > 1 << 24:
                                continue
                            lib.last_place(SMS, batch, heads, group, tokens, queries, context, window, out)
                            splits, last, space, inside = out
                            assert inside and last < space or splits == 1
                            a = H.query_args(num_q_heads=heads * group, batch=batch, max_queries=queries, num_tokens=tokens,
                                             max_context=context, window=window)
                            got = size(C.addressof(h), C.byref(a))
                            if splits > 1:
                                cut += 1
                                assert got >= counters + (last + 1) * (d * 4 + 8), (batch, queries, tokens, context, window)
                            # 256 rows per SM at most, and the few-row kernel's counters, or what that kernel needs
                            assert got <= counters + SMS * 256 * (d * 4 + 8)
    assert cut > 50


def test_few_rows_of_a_padded_buffer(lib):
    """The calls that wrote behind their workspace: few rows of a large buffer of queries, after long contexts."""
    out = (C.c_int64 * 4)()
    for batch, tokens, queries in ((1, 8192, 83), (2, 4096, 100), (1, 512, 17), (1, 256, 32), (1, 64, 32)):
        lib.last_place(SMS, batch, 8, 8, tokens, queries, 16384, 0, out)
        assert out[0] > 1 and out[3]
        a = H.query_args(num_q_heads=64, batch=batch, max_queries=queries, num_tokens=tokens, max_context=16384)
        assert abi.load().paged_query_workspace_size(C.addressof(pool(abi.KV_F16, 128, 8)), C.byref(a)) >= \
            (out[1] + 1) * (128 * 4 + 8)


@pytest.mark.parametrize("dtype", [abi.KV_F32, abi.KV_F16, abi.KV_FP8_E4M3, abi.KV_INT4])
def test_a_size_serves_every_smaller_call(lib, dtype):
    """No call of fewer sequences, rows, rows per sequence or positions needs more, whichever kernel it takes."""
    heads, group = 4, 4
    h = pool(dtype, 128, heads)

    def size(batch, queries, tokens, context, window):
        a = H.query_args(num_q_heads=heads * group, batch=batch, max_queries=queries, num_tokens=tokens, max_context=context,
                         window=window)
        return abi.load().paged_query_workspace_size(C.addressof(h), C.byref(a))

    batches, rows, contexts = (1, 2, 8, 40), (1, 4, 5, 32, 300, 2000), (16, 600, 1023, 1024, 1600, 9000, 70000)
    shapes = [(b, q, t, c) for b in batches for q in rows for t in sorted({q, b * q, b * q + 3, 4 * b * q}) for c in contexts]
    for window in (0, 900):
        largest = {s: size(*s, window) for s in shapes}
        assert min(largest.values()) >= 256
        for s, n in largest.items():
            for i in range(4):                                 # one argument less, and all of them
                for less in (1, s[i] // 2, s[i] - 1):
                    t = s[:i] + (max(less, 1),) + s[i + 1:]
                    if t[1] <= t[2]:
                        assert size(*t, window) <= n, (s, t, window)
            t = tuple(max(x // 3, 1) for x in s)
            if t[1] <= t[2]:
                assert size(*t, window) <= n
            if window == 0:
                assert size(*s, 500) <= n and size(*s, 5000) <= n
