"""Paged attention of a batch that is padded behind its requests' tokens: one request is treated as several are."""
import math

import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16, F16, _attend, _paged

pytestmark = pytest.mark.gpu

PADDED = [
    # dtype, e4m3, dim, kv heads, group, window, new tokens, kv lengths, padding
    (BF16, False, 128, 2, 4, 0, [3], [40], 2),           # few rows with and without the padding
    (BF16, False, 128, 2, 4, 0, [3], [3000], 60),        # few rows, many with the padding; keys divided
    (F16, False, 64, 1, 7, 0, [70], [333], 31),
    (BF16, True, 128, 1, 4, 50, [50], [2500], 300),
    (F16, True, 256, 1, 2, 0, [1], [900], 7),
    (BF16, False, 64, 1, 2, 0, [0], [100], 5),           # no tokens but the padding
    (BF16, False, 128, 1, 4, 0, [2, 5], [90, 5], 40),    # two requests
    (F16, False, 64, 2, 2, 20, [100, 1], [700, 80], 9),
]


@pytest.mark.parametrize("case", PADDED, ids=str)
def test_padding_behind_the_tokens(case):
    dtype, e4m3, D, H, G, window, new, lens, padding = case
    s = _paged(sum(lens) + D, dtype, e4m3, D, H, G, 16, new, lens)
    n = sum(new)
    # each request by itself, without offsets
    want = []
    for b, (t0, t1) in enumerate(zip(s["cu"].tolist(), s["cu"].tolist()[1:])):
        alone = dict(s, q=s["q"][t0:t1], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1], equal=True)
        want.append(_attend(alone, window))
    want = [torch.cat(x) for x in zip(*want)]
    s["q"] = torch.cat([s["q"], torch.full((padding, H * G, D), math.nan, dtype=dtype)])
    out = torch.full_like(s["q"], 7.0).cuda()
    for more in ({}, {"max_q_len": max(new)}) if max(new) else ({},):
        got, lse = _attend(s, window, out=out, **more)
        assert got.data_ptr() == out.data_ptr() and (out[n:] == 7.0).all()
        # kernels and splits go by the tokens that there may be: the same but for roundings, of P (fewer rows: none) and out
        eps = torch.finfo(torch.bfloat16 if e4m3 else dtype).eps
        size = 1 + want[0].double().abs().amax() if n else 1.0
        assert ((got[:n].double() - want[0].double()).abs() <= 2 * eps * size).all()
        # sums of up to 256 products, each side's off by as many fp32 steps of some 15
        assert torch.allclose(lse[:n], want[1], rtol=0, atol=2 * 264 * 2.0 ** -24 * 20)
