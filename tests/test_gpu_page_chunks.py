"""Chunks over caches of 8-bit codes with one scale for each page and head: what a chunk may take from other requests' pages,
and how exactly it has its own."""
import math

import pytest
import torch

from gpu_support import lib  # noqa: F401
from test_gpu_page_scales import _coded, _compare
from test_gpu_serving import BF16, F16, _attend

pytestmark = pytest.mark.gpu


def _one(s, b):
    a, e = int(s["cu"][b]), int(s["cu"][b + 1])
    return dict(s, q=s["q"][a:e], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1], cu=torch.tensor([0, e - a], dtype=torch.int32))


@pytest.mark.parametrize("kind,dtype,dim", [("int8", BF16, 128), ("e4m3", BF16, 128), ("int8", BF16, 64), ("e4m3", BF16, 256),
                                            ("int8", F16, 128)])
@pytest.mark.parametrize("page_0", [math.nan, math.inf, -0.3, 3e38])
def test_a_page_that_is_none_takes_no_scale(kind, dtype, dim, page_0):
    """Zeros in the place of a page outside of the pool, whatever the scale of the first page, which is another request's."""
    s = _coded(dim + 1, kind, dtype, dim, 2, 4, 16, [80, 70], [300, 200], extra=1)
    mine = 1 if 0 in s["table"][0].tolist() else 0  # the request that does not hold page 0
    s["table"][mine, 3] = 2 ** 30
    s["table"][mine, 11] = -1
    want = _attend(s, max_q_len=80)
    for x in "kv":
        s[x + "_scale"][0] = page_0
    got = _attend(s, max_q_len=80)
    a, e = int(s["cu"][mine]), int(s["cu"][mine + 1])
    assert torch.equal(got[0][a:e], want[0][a:e]) and torch.equal(got[1][a:e], want[1][a:e])
    _compare(_one(s, mine), (got[0][a:e], got[1][a:e]), 0, (e - a) * 4)
