"""Chunks over caches of 8-bit codes with one scale for each page and head: what a chunk may take from other requests' pages,
and how exactly it has its own."""
import math

import pytest
import torch

import drafts_oracle as do
import serving_oracle as so
from test_gpu_page_scales import _coded, _compare
from test_gpu_serving import BF16, F16, _attend, _close

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


def _exact_compare(s, got, window, what):
    """Against the form in 64 bits, bf16 queries and codes under powers of two: nothing is rounded to 16 bits but P, to
    fp16's 11 bits (half a step 2^-11; below 2^-14 2^-25, where its row's largest is 2^10 at least), and the output."""
    k, v = (do.values(s[x], s["kind"]) * s[x + "_scale"].double()[:, :, None, None] for x in "kv")
    out, lse, mass, move = so.attention(s["q"], k, v, s["table"], s["kv_len"], s["cu"], s["D"] ** -0.5, window)
    move = move + 4 * so.U32 * (1 + lse.abs().nan_to_num(posinf=0.0))
    ob, lb = so.attention_bounds(out, lse, mass, move, BF16, so.half_step(F16))
    ob = ob + int(s["kv_len"].max()) * 2.0 ** -35 * float((v.abs() * v.isfinite()).nan_to_num(0.0).max())
    _close(got[0], out, ob, what)
    empty = lse == -math.inf
    assert torch.equal(got[1].cpu() == -math.inf, empty) and (got[0].cpu()[empty] == 0).all()
    _close(torch.where(empty, 0.0, got[1].double().cpu()), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


DIGITS = [
    # kind, dim, kv heads, group, page, window, new tokens, kv lengths
    ("int8", 128, 2, 4, 16, 0, [300], [300]),          # rows that see few keys, whose weights' roundings do not average out
    ("e4m3", 128, 2, 4, 16, 0, [300], [300]),
    ("int8", 128, 1, 8, 64, 0, [260, 1, 40], [900, 70, 45]),
    ("e4m3", 128, 1, 1, 8, 5, [200], [333]),
    ("int8", 64, 3, 2, 32, 0, [150, 33], [150, 2500]),
    ("e4m3", 64, 1, 5, 8, 100, [97], [1000]),
    ("int8", 256, 1, 3, 16, 0, [90], [91]),
    ("e4m3", 256, 1, 2, 128, 0, [130], [600]),
    ("int8", 128, 1, 4, 16, 0, [70], [6000]),          # keys divided between workgroups
]


@pytest.mark.parametrize("case", DIGITS, ids=str)
@pytest.mark.parametrize("octaves", [0, 8])
def test_digits_of_weights(case, octaves):
    """Scales that differ by up to `octaves` from page to page, the ends among them, and pages of zeros."""
    kind, D, H, G, page, window, new, lens = case

    def scales(shape, g):
        x = torch.exp2(torch.randint(0, octaves + 1, shape, generator=g).float())
        x[0], x[1] = 1.0, 2.0 ** octaves
        return torch.where(torch.rand(shape, generator=g) < 0.1, 0.0, x) if octaves else x

    s = _coded(sum(new) + D + 3, kind, BF16, D, H, G, page, new, lens, scales if octaves else None, extra=1)
    if octaves:  # what all have in common, far from 1
        s["v_scale"] *= 2.0 ** -40
    got = _attend(s, window, max_q_len=max(new))
    for b in range(len(new)):
        a, e = int(s["cu"][b]), int(s["cu"][b + 1])
        if (e - a) * G > 32:
            _exact_compare(_one(s, b), (got[0][a:e], got[1][a:e]), window, (case, b))
    again = _attend(s, window, max_q_len=max(new))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_every_code(kind):
    """Each code under the ends of 8 octaves, one key to a row (a window of 1): the output is the value itself."""
    page, n = 16, 256
    s = _coded(4, kind, BF16, 128, 1, 1, page, [n], [n])
    codes = torch.arange(n)
    s["v"][s["table"][0].long()[codes // page], 0, codes % page] = (codes - 128).to(torch.int8)[:, None] if kind == "int8" else codes.to(torch.uint8)[:, None]
    for low, high in ((-8, 0), (-100, -92), (92, 100), (-126, -118), (0, 9), (-30, 30)):
        s["v_scale"][:] = 2.0 ** low
        s["v_scale"][1::2] = 2.0 ** high
        got = _attend(s, 1, max_q_len=n)[0][:, 0].cpu()
        unit = s["v_scale"][s["table"][0].long()[codes // page], 0].double()
        value = (codes - 128).double() if kind == "int8" else codes.to(torch.uint8).view(torch.float8_e4m3fn).double()
        want = (value * unit).bfloat16()  # exact for e4m3 and int8, but below 2^-126
        same = (got == want[:, None]) | (got.isnan() & want.isnan()[:, None]) | ((value * unit).abs() < 2.0 ** -126)[:, None]
        assert same.all(), (low, high, codes[~same.all(-1)].tolist())


def test_far_scales_beside_near_ones():
    """A request whose scales lie more than 10 octaves apart, or are no powers of two, beside one whose do not."""
    s = _coded(9, "int8", BF16, 128, 2, 4, 16, [100, 100, 100], [400, 400, 400])
    want = _attend(s, max_q_len=100)
    s["v_scale"][s["table"][0, 2].long()] *= 2.0 ** 12
    s["v_scale"][s["table"][2, 2].long()] *= 1.25
    got = _attend(s, max_q_len=100)
    assert torch.equal(got[0][100:200], want[0][100:200])
    for b in (0, 2):
        _compare(_one(s, b), (got[0][100 * b:100 * b + 100], got[1][100 * b:100 * b + 100]), 0, 400)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_small_weights_of_many_keys(kind, dim):
    """A key whose value is 0 outweighs all others by 2^20 to 2^34, which the output is made of: powers of two, which fp16
    holds down to 2^-24 of weights that are 2^10 at their row's largest, so that nothing but the output is rounded."""
    page, new, length = 16, 60, 3000
    s = _coded(7, kind, BF16, dim, 1, 1, page, [new], [length])
    one = 64 if kind == "int8" else 0x78  # 64 * 2^-6, 256 * 2^-8: 1
    unit = 2.0 ** -6 if kind == "int8" else 2.0 ** -8
    s["q"].zero_()
    far = torch.arange(new) % 15 + 20  # powers of two below the first key
    s["q"][:, 0, 0] = far.to(BF16)
    for x in "kv":
        s[x].zero_()
        s[x + "_scale"][:] = unit
    s["k"][..., 0] = -64 if kind == "int8" else one | 0x80  # -1: a score of -far
    s["v"][:] = one
    p = int(s["table"][0, 0])
    s["k"][p, 0, 0], s["v"][p, 0, 0] = 0, 0
    got = _attend(s, scale=math.log(2.0), max_q_len=new)[0].double().cpu()[:, 0]
    others = (torch.arange(length - new, length)).double() * torch.exp2(-far.double())
    want = (others / (1 + others))[:, None]
    # scores of up to 34 are off by a few fp32 steps each, and so weights by 34 times as much of themselves
    assert ((got - want).abs() <= want * (so.half_step(BF16) + 64 * 34 * so.U32)).all(), (got[:, 0] / want[:, 0] - 1).abs().max()
