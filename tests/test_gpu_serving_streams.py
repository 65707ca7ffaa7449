"""Serving calls on the stream that they are given, by object or by handle."""
import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16, _attend, _paged

pytestmark = pytest.mark.gpu


def test_the_stream_that_is_current_within():
    from hashed_gram_memory_amd import serving
    x = torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    for given, handle in ((0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
        with torch.cuda.stream(torch.cuda.Stream()), serving._on(given, x):
            assert torch.cuda.current_stream().cuda_stream == handle


def test_the_default_stream_by_its_handle():
    """Behind work of the default stream that takes a while, with nothing waited for between."""
    hg = lib()
    s = _paged(15, BF16, False, 128, 2, 4, 16, [1, 1], [300, 40], equal=True)
    want = _attend(s, lse=False)
    args = {k: s[k].cuda() for k in ("q", "k", "v", "table", "kv_len")}
    q = torch.zeros_like(args["q"])
    big = torch.ones(1 << 28, device="cuda")
    torch.cuda.synchronize()
    for _ in range(8):
        big.mul_(1.0)
    q.copy_(args["q"])
    assert torch.cuda.current_stream().cuda_stream == 0
    got = hg.paged_attention(q, args["k"], args["v"], args["table"], args["kv_len"], stream=0)
    turned, _ = hg.qk_norm_rope(got, None, stream=0)
    assert torch.equal(got, want) and torch.equal(turned, want)
