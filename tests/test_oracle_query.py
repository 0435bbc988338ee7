"""Pins of the oracle's query attention: closed forms, the one-token form and torch in float64."""

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import query as OQ


def data(n, c, hq, h, d, seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n, hq, d)), rng.standard_normal((c, h, d)), rng.standard_normal((c, h, d))


def test_one_token_is_decode_attention():
    q, k, v = data(1, 9, 4, 2, 8)
    assert np.allclose(OQ.query_attention(q, k, v, 0.3)[0], OA.decode_attention_gqa(q, [k], [v], 0.3)[0], atol=1e-14)
    assert np.allclose(OQ.query_attention(q, k, v, 0.3, window=4)[0],
                       OA.decode_attention_window(q, [k], [v], 0.3, 4)[0], atol=1e-14)


def test_whole_prompt_is_the_causal_recompute():
    q, k, v = data(7, 7, 1, 1, 8)
    assert np.allclose(OQ.query_attention(q, k, v, 0.5)[:, 0], OA.causal_attention(q[:, 0], k[:, 0], v[:, 0], 0.5),
                       atol=1e-14)


@pytest.mark.parametrize("cap,bias,window", [(0.0, False, 0), (2.0, False, 0), (0.0, True, 3), (1.5, True, 2)])
def test_against_torch(cap, bias, window):
    n, c, hq, h = 5, 11, 4, 2
    q, k, v = data(n, c, hq, h, 8, 3)
    ranges = np.array([[0, 7], [2, 20], [5, 5], [-3, 9], [9, 4]])
    slopes = np.array([0.5, 0.25, 0.1, 0.7]) if bias else None
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    x = torch.einsum("nhd,chd->hnc", tq, tk.repeat_interleave(2, 1)) * 0.7
    if cap:
        x = cap * torch.tanh(x / cap)
    p, j = torch.arange(c - n, c)[:, None], torch.arange(c)[None]
    if bias:
        x = x - torch.from_numpy(slopes)[:, None, None] * (p - j).abs()
    r = torch.from_numpy(ranges)
    seen = (j >= r[:, :1]) & (j < r[:, 1:])
    if window:
        seen &= p - j < window
    w = torch.softmax(x.masked_fill(~seen, -torch.inf), -1).nan_to_num(0.0)
    want = torch.einsum("hnc,chd->nhd", w, tv.repeat_interleave(2, 1))
    got = OQ.query_attention(q, k, v, 0.7, window, cap, slopes, ranges)
    assert np.allclose(got, want.numpy(), atol=1e-13)
    assert not got[2].any() and not got[4].any()


def test_closed_forms():
    q, k, v = data(3, 3, 2, 2, 8)
    assert np.allclose(OQ.query_attention(q, k, v, 1.0)[0], v[0])                # the first row sees one key
    assert np.allclose(OQ.query_attention(0 * q, k, v, 1.0)[2], v.mean(0))       # equal scores
    two = OQ.query_attention(0 * q, k, v, 1.0, slopes=[np.log(3.0)] * 2)[1]      # weights 3 : 1
    assert np.allclose(two, 0.25 * v[0] + 0.75 * v[1])
    big = OQ.query_attention(1e4 * q, k, v, 1.0, cap=1e-9)[2]                    # everything capped to nothing
    assert np.allclose(big, v.mean(0), atol=1e-7)
    seen = OQ.query_attention(q, np.where(np.arange(3)[:, None, None] == 2, np.nan, k), v, 1.0)
    assert np.isfinite(seen[:2]).all() and np.isnan(seen[2]).all()               # what is masked does not reach a row
