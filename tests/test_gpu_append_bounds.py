"""Appends to caches of 8-bit codes with one scale for each page and head: bounds of tokens that requests pass, and scales that
the append itself would not have written."""
import pytest
import torch

import drafts_oracle as do
from gpu_support import lib  # noqa: F401
from test_gpu_append_pages import _batch, _call, _compare, _device
from test_gpu_serving import BF16, F16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dtype,D,R,norm", [("int8", BF16, 128, 0, False), ("e4m3", F16, 64, 0, False), ("int8", BF16, 256, 256, True)])
def test_tokens_past_the_bound(kind, dtype, D, R, norm):
    """max_q_len 1, requests with more: the first token of each is appended (the others may be left out, and here are)."""
    new, lens = [1, 2, 0, 5, 1, 3, 9], [1, 2, 7, 40, 16, 2, 17]
    s = _batch(D, kind, dtype, D, 3, 8, new, lens, R=R, norm=norm)
    d = _device(s)
    _call(d, max_q_len=1)
    first = [int(s["cu"][b]) for b, n in enumerate(new) if n]
    one = dict(s, kv=s["kv"][first], positions=s["positions"][first], cu=torch.tensor([min(n, 1) for n in [0] + new]).cumsum(0).int(),
               # the length up to the first token; tokens before the first key are left out
               kv_len=torch.tensor([max(length - n + 1, 0) if n else length for n, length in zip(new, lens)], dtype=torch.int32))
    _compare(one, d, "the first tokens")


@pytest.mark.parametrize("bound", [2, 3, 7])
def test_a_bound_of_some_tokens(bound):
    """A request with more than max_q_len tokens has those up to it in the cache, on whatever pages they lie."""
    new, lens = [20, 1, 9, 33], [25, 1, 9, 100]
    s = _batch(bound, "int8", BF16, 64, 2, 8, new, lens)
    d = _device(s)
    _call(d, max_q_len=bound)
    for x, cols in (("k", slice(0, 2)), ("v", slice(2, 4))):
        value = do.values(d[x + "_cache"].cpu(), "int8")
        scale = d[x + "_scale"].cpu().double()
        for b, (n, length) in enumerate(zip(new, lens)):
            for i in range(min(n, bound)):
                key = length - n + i
                p = int(s["table"][b, key // 8])
                want = s["kv"][int(s["cu"][b]) + i, cols].double()
                assert ((value[p, :, key % 8] * scale[p][:, None] - want).abs() <= scale[p][:, None] / 2).all(), (x, b, i)
