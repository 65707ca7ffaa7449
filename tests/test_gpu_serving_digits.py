"""Chunks over an e4m3 cache, each type of query held to its own digits; tables much wider than the requests."""
import math

import pytest
import torch

import serving_oracle as so
from test_gpu_serving import BF16, F16, _attend, _close, _paged

pytestmark = pytest.mark.gpu

CHUNKS = [
    # dtype, dim, kv heads, group, page, window, new tokens, kv lengths, columns of the table past the longest request
    (F16, 64, 1, 5, 16, 0, [77], [300], 0),
    (F16, 64, 2, 2, 8, 100, [200, 1, 40], [900, 700, 40], 3),
    (F16, 128, 2, 4, 32, 0, [70, 3], [513, 40], 1),
    (F16, 128, 1, 2, 128, 0, [257], [4100], 0),          # divided
    (F16, 128, 6, 4, 16, 0, [9] * 50, [90] * 50, 0),     # half tiles
    (F16, 256, 1, 3, 8, 40, [50], [129], 0),
    (F16, 256, 2, 1, 16, 0, [33, 70], [1500, 70], 0),
    (BF16, 256, 1, 4, 16, 0, [40, 90], [700, 90], 0),
    (BF16, 256, 2, 2, 64, 333, [150], [2000], 2),
    (BF16, 128, 1, 8, 8, 0, [64], [1000], 4000),
    (F16, 64, 1, 8, 8, 0, [30, 5], [1000, 30], 4000),
]


@pytest.mark.parametrize("case", CHUNKS, ids=str)
def test_e4m3_chunks(case):
    dtype, D, H, G, page, window, new, lens, extra = case
    s = _paged(sum(new) + D + page, dtype, True, D, H, G, page, new, lens, extra=extra)
    out, lse, mass, move = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], D ** -0.5, window,
                                        s["k_scale"], s["v_scale"])
    ob, lb = so.attention_bounds(out, lse, mass, move, dtype, so.half_step(dtype))
    # the product of P and V's scale is rounded in fp32; an fp16 P is held with its row's largest at 2^7 or more, so that
    # below 2^-14 it is off by 2^-32 of that largest at most
    ob = ob + 4 * so.U32 * mass
    if dtype == F16:
        ob = ob + max(lens) * 2.0 ** -32 * 448 * float(s["v_scale"][s["v_scale"].isfinite()].max())
    got = _attend(s, window, max_q_len=max(new))
    _close(got[0], out, ob, "out")
    empty = lse == -math.inf
    assert torch.equal(got[1].cpu() == -math.inf, empty)
    _close(torch.where(empty, 0.0, got[1].double().cpu()), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


@pytest.mark.parametrize("dtype,e4m3,D", [(BF16, False, 128), (F16, False, 64), (BF16, False, 256), (F16, True, 128)], ids=str)
@pytest.mark.parametrize("new", [[64], [1], [20, 90, 1, 5]], ids=str)
def test_wide_tables(dtype, e4m3, D, new):
    """A table for the longest context that a server allows: the keys are divided by its width, the results are the same
    but for roundings."""
    lens = [4096, 700, 333, 90][:len(new)]
    s = _paged(sum(new) + D, dtype, e4m3, D, 1, 4, 16, new, lens)
    near = _attend(s, max_q_len=max(new))
    wide = torch.full((len(new), 8192), -1, dtype=torch.int32)
    wide[:, :s["table"].shape[1]] = s["table"]
    far = _attend(dict(s, table=wide), max_q_len=max(new))
    out, lse, mass, move = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], D ** -0.5, 0,
                                        s["k_scale"], s["v_scale"])
    ob, lb = so.attention_bounds(out, lse, mass, move, dtype, so.half_step(BF16 if e4m3 else dtype))
    if dtype == F16:
        ob = ob + max(lens) * 2.0 ** -32 * float(s["v"].view(torch.float8_e4m3fn).float().nan_to_num().abs().max() if e4m3
                                                else s["v"][s["v"].isfinite()].abs().max())
    for got in (near, far):
        _close(got[0], out, ob, "out")
        _close(got[1], lse, lb, "lse")
