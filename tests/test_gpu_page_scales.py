"""Paged attention over caches of 8-bit codes with one scale for each page and head, against the plain form in 64 bits."""
import math

import pytest
import torch

import drafts_oracle as do
import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, F16, P_SPLIT, _attend, _close, _paged

pytestmark = pytest.mark.gpu


def _coded(seed, kind, dtype, D, H, G, page, q_lens, kv_lens, scales=None, **more):
    """A batch as in the other caches' tests, its cache as codes; NaN (e4m3) or the largest code in places that no request
    holds, and NaN as the scale of pages of which it holds nothing."""
    s = _paged(seed, dtype, False, D, H, G, page, q_lens, kv_lens, **more)
    g = torch.Generator().manual_seed(seed + 1)
    for x in "kv":
        r = s[x].float()
        hole = r.isnan()
        r = r.nan_to_num(0.0)
        scale = do.power_of_two(r.abs().amax((2, 3)) / do.LARGEST[kind]).float()
        if scales is not None:
            scale = scale * scales(scale.shape, g)
        unit = torch.where(scale > 0, scale, 1.0)[:, :, None, None]
        if kind == "int8":
            codes = (r / unit).round().clamp(-127, 127).to(torch.int8)
            codes[hole] = -128
        else:
            codes = (r / unit).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[hole] = 0x7F
        scale[hole.all(-1).all(-1)] = math.nan
        s[x], s[x + "_scale"] = codes, scale
    s["kind"] = kind
    return s


def _compare(s, got, window, rows, scale=None, extra=0.0):
    """rows: of the longest request; up to 32 P is held in about 16 bits (as bf16 and remainder), else rounded once to q's type.
    A product with a scale that is no power of two is one rounding of fp32 more, on either side."""
    scale = s["D"] ** -0.5 if scale is None else scale
    k, v = (do.values(s[x], s["kind"]) * s[x + "_scale"].double()[:, :, None, None] for x in "kv")
    if rows > 32 and s["dtype"] == BF16:  # the numbers that codes stand for are bf16's there: exact for a power of two
        k, v = ((do.values(s[x], s["kind"]).float() * s[x + "_scale"][:, :, None, None]).bfloat16().double() for x in "kv")
    out, lse, mass, move = so.attention(s["q"], k, v, s["table"], s["kv_len"], s["cu"], scale, window)
    move = move + 4 * so.U32 * (1 + lse.abs().nan_to_num(posinf=0.0))
    step = P_SPLIT[BF16] if rows <= 32 else so.half_step(s["dtype"])
    ob, lb = so.attention_bounds(out, lse, mass, move, s["dtype"], step)
    if rows > 32 and s["dtype"] == F16:
        # P times V's scale is held with its row's largest at 2^7 or more: below 2^-14 it is off by 2^-32 of that at most
        top = float((v.abs() * v.isfinite()).nan_to_num(0.0).max())
        ob = ob + int(s["kv_len"].max()) * 2.0 ** -32 * max(top, 1e-30) * (128 if s["kind"] == "int8" else 448)
    _close(got[0], out, ob + extra, "out")
    l, empty = got[1].double().cpu(), lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert (got[0].cpu()[empty] == 0).all()
    _close(torch.where(empty, 0.0, l), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


CASES = [
    # kind, dtype, dim, kv heads, group, page, window, new tokens, kv lengths
    ("int8", BF16, 128, 1, 1, 16, 0, [1], [1]),
    ("int8", BF16, 128, 8, 4, 16, 0, [1], [512]),
    ("e4m3", BF16, 128, 2, 4, 16, 0, [1] * 13, [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]),
    ("int8", F16, 64, 2, 7, 8, 0, [1] * 3, [5, 1000, 77]),
    ("e4m3", F16, 256, 1, 5, 32, 0, [1] * 2, [999, 64]),
    ("int8", BF16, 256, 2, 1, 1024, 0, [1], [1500]),
    ("int8", BF16, 64, 3, 16, 128, 0, [1] * 2, [130, 1]),
    ("e4m3", BF16, 128, 2, 2, 16, 1, [1] * 3, [40, 1, 0]),
    ("int8", F16, 128, 2, 3, 16, 100, [1] * 4, [50, 100, 101, 5000]),
    ("int8", BF16, 128, 1, 2, 8, 0, [1], [9001]),
    ("int8", BF16, 128, 2, 4, 16, 0, [3, 0, 1, 4, 0], [3, 9, 0, 2, 0]),
    ("e4m3", F16, 64, 1, 4, 32, 20, [4, 3], [1000, 33]),
    ("int8", F16, 256, 1, 3, 8, 33, [6, 2], [200, 10]),
    ("int8", BF16, 128, 2, 4, 16, 0, [70], [200]),
    ("e4m3", F16, 64, 1, 7, 8, 0, [97], [333]),
    ("int8", F16, 256, 1, 2, 32, 0, [130], [157]),
    ("e4m3", BF16, 256, 1, 3, 8, 40, [50], [129]),
    ("int8", BF16, 64, 1, 65, 64, 0, [1], [700]),
    ("int8", F16, 128, 1, 8, 8, 0, [9, 0, 1, 300, 16, 8], [9, 4, 700, 301, 16, 64]),
    ("e4m3", BF16, 128, 1, 2, 128, 0, [257], [4100]),
    ("int8", F16, 64, 3, 1, 16, 0, [100, 200], [50, 200]),
    ("int8", BF16, 128, 2, 1, 16, 333, [300, 1, 90], [900, 1200, 95]),
    ("int8", BF16, 64, 1, 1, 1024, 0, [600], [2100]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(case):
    kind, dtype, D, H, G, page, window, new, lens = case
    s = _coded(sum(new) + D + page, kind, dtype, D, H, G, page, new, lens, extra=1)
    got = _attend(s, window, max_q_len=max(new))
    for b in range(len(new)):  # each request by the form that its rows take
        a, e = int(s["cu"][b]), int(s["cu"][b + 1])
        if a == e:
            continue
        one = dict(s, q=s["q"][a:e], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1],
                   cu=torch.tensor([0, e - a], dtype=torch.int32))
        _compare(one, (got[0][a:e], got[1][a:e]), window, (e - a) * G)
    again = _attend(s, window, max_q_len=max(new))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 50])
def test_any_finite_scale(kind, new):
    """Scales that differ by 2^17 from page to page, are no powers of two, negative or zero."""
    for dtype in (BF16, F16):
        def scales(shape, g):
            x = torch.exp2(torch.randint(-14, 4, shape, generator=g).float()) * (0.5 + torch.rand(shape, generator=g))
            x[torch.rand(shape, generator=g) < 0.1] = 0.0
            return torch.where(torch.rand(shape, generator=g) < 0.3, -x, x)
        s = _coded(new + 5, kind, dtype, 128, 2, 3, 8, [new, 1], [300, 77], scales)
        for x in "kv":  # codes of the whole range, whatever the scale
            g = torch.Generator().manual_seed(9)
            far = s[x] if kind == "int8" else s[x]
            hole = (far == -128) if kind == "int8" else (far == 0x7F)
            any_ = (torch.randint(-127, 128, far.shape, generator=g).to(torch.int8) if kind == "int8"
                    else torch.randint(0, 0x7F, far.shape, generator=g).to(torch.uint8))
            s[x] = torch.where(hole, far, any_)
        k = do.values(s["k"], kind) * s["k_scale"].double()[:, :, None, None]
        s["k_scale"] = (s["k_scale"].double() / k.abs().nan_to_num(0.0).max() * 4).float()
        v = do.values(s["v"], kind) * s["v_scale"].double()[:, :, None, None]
        s["v_scale"] = (s["v_scale"].double() / v.abs().nan_to_num(0.0).max() * 4).float()
        got = _attend(s, max_q_len=new)
        for b in range(2):
            a, e = int(s["cu"][b]), int(s["cu"][b + 1])
            one = dict(s, q=s["q"][a:e], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1],
                       cu=torch.tensor([0, e - a], dtype=torch.int32))
            _compare(one, (got[0][a:e], got[1][a:e]), 0, (e - a) * 3)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [5, 60])
def test_what_is_hidden(kind, new):
    """Pages that are none, pages with a scale of NaN or infinity that no token sees, behind a window and past the end."""
    s = _coded(new, kind, BF16, 128, 2, 4, 16, [new, 2], [200, 45])
    window = 70
    clean = _attend(s, window, max_q_len=new)
    first = (200 - new + 1 - window) // 16  # pages before it are seen by no token
    assert first > 0
    for p in s["table"][0, :first]:
        for x in "kv":
            s[x + "_scale"][int(p)] = math.inf if int(p) % 2 else math.nan
    dirty = _attend(s, window, max_q_len=new)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    s["table"][0, :first] = -1
    s["table"][0, first + 2] = 2 ** 31 - 1
    s["table"][1, 0] = s["k"].shape[0]
    got = _attend(s, window, max_q_len=new)
    for b, n in enumerate((new, 2)):
        a, e = int(s["cu"][b]), int(s["cu"][b + 1])
        one = dict(s, q=s["q"][a:e], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1], cu=torch.tensor([0, n], dtype=torch.int32))
        _compare(one, (got[0][a:e], got[1][a:e]), window, n * 4)


@pytest.mark.parametrize("new", [1, 40])
def test_a_scale_of_nan_is_seen(new):
    """By the tokens that see a row of its page, and by those alone."""
    s = _coded(3, "int8", BF16, 64, 1, 2, 8, [new, 1], [64, 20])
    s["v_scale"][int(s["table"][0, 7]), 0] = math.nan  # keys 56 to 63
    out, lse = _attend(s, max_q_len=new)
    sees = torch.arange(64 - new, 64) >= 56
    assert torch.equal(out[:new].isnan().any(-1).any(-1).cpu(), sees) and out[new:].isfinite().all() and lse.isfinite().all()


SETS = [
    # kind, dtype, dim, kv heads, group, page, window, new tokens, kv lengths: 17 to 32 rows of a request, and fewer beside them
    ("int8", BF16, 128, 8, 4, 16, 0, [6] * 3, [700, 6, 33]),
    ("e4m3", BF16, 128, 2, 4, 32, 0, [6, 1, 0, 8, 4, 5], [3000, 40, 7, 8, 128, 4]),
    ("int8", F16, 64, 2, 17, 8, 0, [1, 1], [999, 17]),
    ("e4m3", F16, 64, 3, 5, 16, 40, [5, 6, 2], [300, 41, 39]),
    ("int8", BF16, 256, 1, 8, 64, 0, [4, 3], [2500, 100]),
    ("e4m3", F16, 256, 2, 3, 8, 100, [10, 7], [64, 1000]),
    ("int8", BF16, 128, 1, 32, 16, 0, [1] * 5, [5000, 1, 0, 250, 129]),
    ("int8", BF16, 64, 1, 1, 16, 0, [32, 17, 20], [9000, 17, 40]),
]


@pytest.mark.parametrize("case", SETS, ids=str)
def test_two_sets_of_rows(case):
    kind, dtype, D, H, G, page, window, new, lens = case
    s = _coded(sum(new) + D + page, kind, dtype, D, H, G, page, new, lens, extra=1)
    got = _attend(s, window, max_q_len=max(new))
    _compare(s, got, window, 32)
    again = _attend(s, window, max_q_len=max(new))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    # one request by itself, whose rows the host knows
    a, e = int(s["cu"][0]), int(s["cu"][1])
    one = dict(s, q=s["q"][a:e], table=s["table"][:1], kv_len=s["kv_len"][:1], cu=s["cu"][:2], equal=True)
    _compare(one, _attend(one, window), window, 32)


@pytest.mark.parametrize("dim,group,new", [(128, 4, 6), (64, 2, 5), (256, 3, 9), (128, 4, 40)])
def test_a_code_of_nan_is_seen(dim, group, new):
    """By the tokens that see its key, in K and in V, in either set of rows; the others' results are what they would be."""
    s = _coded(new + dim, "e4m3", BF16, dim, 2, group, 16, [new, 1], [150, 20])
    for x in "kv":
        bad = dict(s, **{x: s[x].clone()})
        key = 150 - new + new // 2
        bad[x][int(s["table"][0, key // 16]), 1, key % 16, 3] = 0x7F
        out, lse = _attend(bad, max_q_len=new)
        sees = torch.zeros(new + 1, 2 * group, dtype=torch.bool)
        sees[new // 2:new, group:] = True
        nan = sees[..., None].expand(out.shape).clone()
        if x == "v":
            nan[..., :3] = nan[..., 4:] = False
            sees[:] = False
        assert torch.equal(out.isnan().cpu(), nan) and torch.equal(lse.isnan().cpu(), sees)
        # Against the form without the NaN where it does not reach.  (Not bit by bit against a call without it: V's products
        # of a step that holds a NaN are added key by key, each within what _compare allows for P's two parts.)
        k, v = (do.values(s[y], "e4m3") * s[y + "_scale"].double()[:, :, None, None] for y in "kv")
        want, want_lse, _, _ = so.attention(s["q"], k, v, s["table"], s["kv_len"], s["cu"], dim ** -0.5, 0)
        for b in range(2):
            a, e = int(s["cu"][b]), int(s["cu"][b + 1])
            one = dict(s, q=s["q"][a:e], table=s["table"][b:b + 1], kv_len=s["kv_len"][b:b + 1], cu=torch.tensor([0, e - a], dtype=torch.int32))
            mended = torch.where(nan[a:e], want[a:e], out[a:e].double().cpu()), torch.where(sees[a:e], want_lse[a:e], lse[a:e].double().cpu())
            _compare(one, mended, 0, (e - a) * group)
