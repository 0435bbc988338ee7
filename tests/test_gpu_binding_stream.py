"""GPU: the stream that the binding passes on."""

import pytest
import torch

from paged_kv_cache_169_gb300 import cache as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("private", [True, False])
def test_the_current_stream_by_either_way(monkeypatch, private):
    if not private:
        monkeypatch.setattr(C, "_raw_stream", None)
    assert C._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert C._stream(None) == side.cuda_stream
    assert C._stream(side) == side.cuda_stream
    cache = C.PagedKVCache(1, 4, 16, 2, 64, "f16")
    k = torch.randn(5, 2, 64, device="cuda").half()
    slots = torch.arange(5, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):                      # one after the other on the current stream
        for _ in range(20):
            torch.randn(1024, 1024, device="cuda") @ torch.randn(1024, 1024, device="cuda")
        k.mul_(2)
        cache.append(0, k, k, slots)
        gk, _ = cache.gather(0, slots)
    side.synchronize()
    assert torch.equal(gk, k)
    cache.close()
