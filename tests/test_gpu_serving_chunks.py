"""Paged attention of many rows per request (chunks of prompts) against the plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, F16, _attend, _close, _paged

pytestmark = pytest.mark.gpu


def _compare(s, got, window=0, scale=None):
    """P is rounded once to 16 bits here.  An fp16 P is held with its row's reference at 2^7, so that below 2^-14 it is
    off by 2^-25 at most: 2^-32 of the sum for each key."""
    scale = s["D"] ** -0.5 if scale is None else scale
    out, lse, mass, move = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], scale, window,
                                        s["k_scale"], s["v_scale"])
    p_type = BF16 if s["k_scale"] is not None else s["dtype"]
    ob, lb = so.attention_bounds(out, lse, mass, move, s["dtype"], so.half_step(p_type))
    if p_type == F16:
        ob = ob + int(s["kv_len"].max()) * 2.0 ** -32 * float(s["v"][s["v"].isfinite()].abs().max())
    _close(got[0], out, ob, "out")
    l = got[1].double().cpu()
    empty = lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert (got[0].cpu()[empty] == 0).all()
    _close(torch.where(empty, 0.0, l), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


CHUNKS = [
    # dtype, e4m3, dim, kv heads, group, page, window, new tokens, kv lengths
    (BF16, False, 128, 1, 1, 16, 0, [65], [65]),                     # a prompt's start: the first rows see few keys
    (BF16, False, 128, 2, 4, 16, 0, [70], [200]),
    (F16, False, 64, 1, 7, 8, 0, [97], [333]),
    (F16, False, 256, 1, 2, 32, 0, [130], [157]),
    (BF16, False, 64, 1, 65, 64, 0, [1], [700]),                     # one token with a group of many heads
    (BF16, False, 128, 1, 8, 8, 0, [9, 0, 1, 300, 16, 8], [9, 4, 700, 301, 16, 64]),  # long and short runs in one call
    (BF16, False, 128, 1, 2, 128, 0, [257], [4100]),                 # few rows, many keys: divided
    (F16, False, 64, 3, 1, 16, 0, [100, 200], [50, 200]),            # rows before the first key
    (BF16, False, 128, 1, 4, 16, 50, [80], [400]),                   # windows below, at and above the tile's keys
    (F16, False, 64, 2, 3, 16, 64, [150, 40], [1000, 40]),
    (BF16, False, 256, 1, 1, 16, 1, [140], [150]),
    (BF16, False, 128, 2, 1, 16, 333, [300, 1, 90], [900, 1200, 95]),
    (BF16, True, 128, 2, 4, 32, 0, [70, 3], [513, 40]),
    (F16, True, 64, 1, 5, 16, 0, [77], [300]),
    (F16, True, 256, 1, 3, 8, 40, [50], [129]),
    (BF16, True, 64, 1, 1, 1024, 0, [600], [2100]),
]


@pytest.mark.parametrize("case", CHUNKS, ids=str)
def test_attention_chunks(case):
    dtype, e4m3, D, H, G, page, window, new, lens = case
    s = _paged(sum(new) + D + page, dtype, e4m3, D, H, G, page, new, lens, extra=1)
    got = _attend(s, window, max_q_len=max(new))
    _compare(s, got, window)
    # without the bound, and on every call: the same bits
    again = _attend(s, window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype,e4m3,D", [(BF16, False, 128), (F16, False, 64), (BF16, True, 128), (F16, True, 256)], ids=str)
def test_chunks_hide_what_is_masked(dtype, e4m3, D):
    """NaN and infinities in keys and values that a token may not see change nothing."""
    n, length = 90, 150
    s = _paged(5, dtype, e4m3, D, 1, 2, 8, [n], [length])
    clean = _attend(s)
    _compare(s, clean)
    at = 120  # seen by the tokens 60 and later
    page, place = int(s["table"][0, at // 8]), at % 8
    if e4m3:
        s["k"][page, 0, place, 3] = 0x7F
        s["v"][page, 0, place, 9] = 0xFF
    else:
        s["k"][page, 0, place, 3] = math.inf
        s["v"][page, 0, place, 9] = -math.inf
        s["v"][page, 0, place, 37] = math.nan
    got = _attend(s)
    assert got[0][60:].isnan().any(-1).all()
    hidden = dict(s, q=s["q"][:60], cu=torch.tensor([0, 60], dtype=torch.int32),
                  kv_len=torch.tensor([120], dtype=torch.int32))
    _compare(hidden, (got[0][:60], got[1][:60]))
    # only values: keys are finite, so that the hidden value meets a weight of zero
    s = _paged(6, dtype, e4m3, D, 1, 2, 8, [n], [length])
    page, place = int(s["table"][0, 100 // 8]), 100 % 8
    if e4m3:
        s["v_scale"][page, 0, place] = math.nan
    else:
        s["v"][page, 0, place, ::3] = math.nan
    got = _attend(s)
    assert got[0][40:].isnan().any(-1).all() and got[1].isfinite().all()
    hidden = dict(s, q=s["q"][:40], cu=torch.tensor([0, 40], dtype=torch.int32),
                  kv_len=torch.tensor([100], dtype=torch.int32))
    _compare(hidden, (got[0][:40], got[1][:40]))
    # a window hides the oldest keys in the same way
    s = _paged(7, dtype, e4m3, D, 1, 2, 8, [n], [length])
    page = int(s["table"][0, 2])
    if e4m3:
        s["v"][page, 0, 3] = 0x7F
    else:
        s["v"][page, 0, 3] = math.inf  # key 19: the token at 60 + i sees keys from i + 11 on
    got = _attend(s, window=50)
    assert not got[0][:9].isfinite().all() and got[0][9:].isfinite().all()
    later = dict(s, q=s["q"][9:], cu=torch.tensor([0, n - 9], dtype=torch.int32))
    _compare(later, (got[0][9:], got[1][9:]), window=50)


def test_chunks_skip_pages_outside_the_pool():
    for dtype, e4m3 in ((BF16, False), (BF16, True)):
        s = _paged(9, dtype, e4m3, 64, 1, 2, 8, [100, 70], [150, 80])
        s["table"][0, 2] = -1
        s["table"][0, 15] = 2 ** 31 - 1
        s["table"][1] = -7  # no keys at all
        got = _attend(s)
        _compare(s, got)
        assert (got[0][100:] == 0).all() and (got[1][100:] == -math.inf).all()


def test_chunks_bound_lengths():
    """Lengths below zero and past the table are bounded by what the table holds."""
    s = _paged(10, BF16, False, 64, 1, 2, 8, [80, 80], [96, 96])
    s["kv_len"] = torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32)
    _compare(s, _attend(s))


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_chunks_extreme_scores(dtype):
    """Scores far apart, all equal, very negative, rising and falling along the keys: the reference carries them."""
    s = _paged(12, dtype, False, 64, 1, 2, 16, [70], [600])
    for scale in (0.0, 5.0, -5.0, 1e-6):
        _compare(s, _attend(s, scale=scale), scale=scale)
    length = 600
    for slope in (0.05, -0.05, 3.0, -3.0):  # within the slack of a tile, and far past it
        for j in range(length):
            page = int(s["table"][0, j // 16])
            s["k"][page, :, j % 16] = slope * (j - 300) / 64
        s["q"][:] = 1.0
        _compare(s, _attend(s, scale=1.0), scale=1.0)


def test_chunks_strided_on_another_stream_and_in_a_graph():
    """Slices of one projection's output, a cache of halves of one allocation, given outputs; on another stream; replayed."""
    s = _paged(13, BF16, False, 128, 2, 2, 16, [150, 3, 80], [150, 70, 1100])
    plain = _attend(s)
    T = 233
    packed = torch.zeros((T, 9, 128), dtype=BF16, device="cuda")
    packed[:, 2:6] = s["q"].cuda()
    both = torch.stack([s["k"], s["v"]], 1).cuda()
    table, lens, cu = s["table"].cuda(), s["kv_len"].cuda(), s["cu"].cuda()
    out = torch.full((T, 6, 128), 7.0, dtype=BF16, device="cuda")

    def call(**more):
        return lib().paged_attention(packed[:, 2:6], both[:, 0], both[:, 1], table, lens, cu_q=cu, **more)

    assert torch.equal(call(out=out[:, 1:5]), plain[0]) and (out[:, 0] == 7).all() and (out[:, 5] == 7).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, plain[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    g = torch.Generator().manual_seed(1)
    for _ in range(4):
        packed.copy_(torch.randn(packed.shape, generator=g).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        here = got.clone()
        assert torch.equal(here, call())


def test_a_bound_of_the_runs_chooses_kernels_alone():
    """One token each, by equal lengths, by offsets with and without the bound; a bound below a run leaves other runs as they are."""
    lens = [300, 1, 64, 65]
    s = _paged(3, BF16, False, 64, 2, 4, 16, [1] * 4, lens)
    by_bound, unknown = _attend(s, max_q_len=1), _attend(s)
    s["equal"] = True
    equal = _attend(s)
    assert torch.equal(by_bound[0], equal[0]) and torch.equal(unknown[0], equal[0])
    new = [1, 90, 2]
    s = _paged(4, BF16, False, 64, 1, 4, 16, new, [100, 200, 300])
    whole = _attend(s, max_q_len=90)
    part = _attend(s, max_q_len=2)
    for rows in (slice(0, 1), slice(91, 93)):
        assert torch.equal(whole[0][rows], part[0][rows])


def test_many_requests_of_both_kinds():
    rng = np.random.default_rng(8)
    new = [int(rng.choice([0, 1, 2, 20, 70])) for _ in range(150)]
    lens = [int(rng.integers(n, 120)) for n in new]
    s = _paged(11, F16, False, 64, 1, 2, 8, new, lens)
    _compare(s, _attend(s, max_q_len=70))


MANY = [
    # dtype, e4m3, kv heads, group, page, window, requests, new tokens, longest: more tiles of 256 rows than CUs
    (BF16, False, 8, 4, 16, 0, 40, 9, 150),
    (F16, False, 8, 4, 8, 40, 36, 33, 100),
    (BF16, True, 6, 4, 16, 0, 50, 9, 90),
    (F16, True, 9, 3, 32, 17, 30, 12, 64),
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_attention_of_many_short_chunks(case):
    """Half tiles of head_dim 128; the same requests, the first with infinities and NaN where others end."""
    dtype, e4m3, H, G, page, window, n, new, longest = case
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(new // 2, longest, n)]
    s = _paged(n + page, dtype, e4m3, 128, H, G, page, [new] * n, lens, equal=True)
    _compare(s, _attend(s, window), window)
    ragged = [int(x) for x in rng.integers(9, new + 1, n)]
    s = _paged(n + page + 1, dtype, e4m3, 128, H, G, page, ragged, lens)
    if not e4m3:  # seen by the last token of the first request alone
        at = lens[0] - 1
        where = int(s["table"][0, at // page]), 0, at % page
        s["v"][where][0], s["v"][where][1] = math.inf, math.nan
    got = _attend(s, window)
    if not e4m3:
        last = ragged[0] - 1
        assert got[0][last, :G, 0].isinf().all() and got[0][last, :G, 1].isnan().all()
        assert got[0][:last].isfinite().all() and got[0][last, :, 2:].isfinite().all()
        s["v"][where][:2] = 0.0
        got[0][last, :G, :2] = 0.0
        out = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], 128 ** -0.5, window)[0]
        got[0][last, :G, :2] = out[last, :G, :2].to(dtype).cuda()
    _compare(s, got, window)


@pytest.mark.parametrize("case", [(64, 2, 3, 16, 0, [150, 40], [500, 40]), (128, 1, 4, 32, 0, [70, 9], [300, 700]),
                                  (128, 8, 4, 8, 20, [9] * 40, [64] * 40), (256, 1, 2, 16, 33, [90], [140])], ids=str)
def test_e4m3_weights_keep_the_digits_of_fp16(case):
    """An fp16 P over an e4m3 cache, with scales of V that differ by 2^17 from key to key, are zero, or all far from 1."""
    D, H, G, page, window, new, lens = case
    for far in (0, -24, 20):
        s = _paged(D + page + far, F16, True, D, H, G, page, new, lens)
        g = torch.Generator().manual_seed(D + far)
        by = torch.randint(-14, 4, s["v_scale"].shape, generator=g).double()
        s["v_scale"] = (s["v_scale"].double() * torch.exp2(by + far)).float()
        s["v_scale"][torch.rand(s["v_scale"].shape, generator=g) < 0.05] = 0.0
        if far > 0:
            s["v_scale"] = s["v_scale"].clamp(max=100.0)  # fp16's range
        out, lse, mass, move = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], D ** -0.5, window,
                                            s["k_scale"], s["v_scale"])
        ob, lb = so.attention_bounds(out, lse, mass, move, F16, so.half_step(F16))
        # the product with the scale is rounded in fp32; P is held with its row's largest at 2^7 or more, so that below
        # 2^-14 it is off by 2^-32 of that largest at most
        ob = ob + 4 * so.U32 * mass + max(lens) * 2.0 ** -32 * 448 * float(s["v_scale"][s["v_scale"].isfinite()].max())
        got = _attend(s, window, max_q_len=max(new))
        _close(got[0], out, ob, ("out", far))
        empty = lse == -math.inf
        _close(torch.where(empty, 0.0, got[1].double().cpu()), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


@pytest.mark.parametrize("tokens", [1, 50])
def test_attention_without_keys(tokens):
    """A table of no pages: zeros, and -infinity for lse."""
    q = torch.randn((2 * tokens, 8, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    cache = torch.full((3, 2, 16, 128), math.nan, dtype=BF16, device="cuda")
    table = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    out, lse = lib().paged_attention(q, cache, cache, table, torch.tensor([5, 0], dtype=torch.int32, device="cuda"),
                                     return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
