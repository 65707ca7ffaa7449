"""Appends to caches of 8-bit codes with one scale for each page and head, against the plain form in 64 bits.

Rows that no arithmetic moves are exact: their maxima, quotients by a power of two and codes have no rounding but the one to
the code, so codes and scales are compared bit by bit.  Normed and rotated keys are within drafts_oracle.append's bounds."""
import math

import numpy as np
import pytest
import torch

import drafts_oracle as do
import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, F16, _freq, _gen, _normal

pytestmark = pytest.mark.gpu


def _codes(shape, kind, g):
    """Codes as they may lie in a cache: any number of the kind."""
    if kind == "int8":
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    c = torch.randint(0, 0x7F, shape, generator=g, dtype=torch.uint8)
    return c | torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7


def _batch(seed, kind, dtype, D, H, page, new, lens, R=0, norm=False, interleaved=False, spread=6, spare=2):
    """New tokens of requests over a pool in random order that other numbers fill."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    width = max(need + [1]) + 1
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), width), 2 ** 30, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    T = sum(new)
    kv = _normal((T, 2 * H, D), torch.float32, g) * torch.exp2(torch.randint(-spread, spread + 1, (T, 2 * H, 1), generator=g).float())
    s = {"kind": kind, "dtype": dtype, "kv": kv.to(dtype), "table": torch.from_numpy(table),
         "kv_len": torch.tensor(lens, dtype=torch.int32), "cu": torch.tensor([0] + new).cumsum(0).int(), "H": H,
         "freq": _freq(R) if R else None, "weight": _normal((D,), dtype, g) + 1 if norm else None, "interleaved": interleaved,
         "positions": torch.cat([torch.arange(n - m, n, dtype=torch.int32) for m, n in zip(new, lens)] + [torch.zeros(0).int()])}
    for x in "kv":
        s[x + "_cache"] = _codes((pages, H, page, D), kind, g)
        s[x + "_scale"] = torch.exp2(torch.randint(-spread - 7, spread, (pages, H), generator=g).float())
    return s


def _device(s):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in s.items()}


def _call(d, equal=False, **more):
    H = d["H"]
    lib().kv_append_pages(d["kv"][:, :H], d["kv"][:, H:], d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], d["table"],
                          d["kv_len"], cu_q=None if equal else d["cu"], positions=d["positions"] if d["freq"] is not None else None,
                          inv_freq=d["freq"], k_weight=d["weight"], eps=1e-6, interleaved=d["interleaved"], **more)


def _compare(s, d, what=""):
    """The device's caches after the call against the form's, from the state s before it."""
    H, kind = s["H"], s["kind"]
    k, fp = so.norm_rope(s["kv"][:, :H], s["weight"], 1e-6, s["positions"], s["freq"], s["interleaved"])
    exact = s["weight"] is None and s["freq"] is None
    for x, rows, off in (("k", k, torch.zeros_like(fp) if exact else fp), ("v", s["kv"][:, H:].double(), torch.zeros_like(k))):
        held, scale, bound, low, high = do.append(rows, off, s[x + "_cache"], s[x + "_scale"], s["table"], s["kv_len"], s["cu"], kind)
        got_scale = d[x + "_scale"].cpu().double()
        nan = scale.isnan()
        assert torch.equal(got_scale.isnan(), nan), (what, x, "scales that are NaN")
        assert ((got_scale == low) | (got_scale == high) | nan).all(), (what, x, "scales")
        got, sure = do.values(d[x + "_cache"].cpu(), kind), ~nan[:, :, None, None]
        same = (got_scale == scale)[:, :, None, None] & sure
        plain = same & (bound == 0)
        wrong = plain & (got != held) & ~(got.isnan() & held.isnan())
        assert not wrong.any(), (what, x, int(wrong.sum()))
        fine = ((got * got_scale[:, :, None, None] - held * scale[:, :, None, None]).abs()
                <= bound * torch.maximum(got_scale / scale, torch.ones(1)).nan_to_num(1.0)[:, :, None, None])
        moved = sure & (bound > 0) & ~fine
        assert not moved.any(), (what, x, int(moved.sum()))


CASES = [
    # kind, dtype, dim, heads, page, rotary, norm, interleaved, new tokens, lengths
    ("int8", BF16, 128, 8, 16, 0, False, False, [1], [1]),
    ("int8", BF16, 128, 8, 16, 0, False, False, [1, 1, 1, 1, 1], [16, 17, 33, 40, 8]),
    ("e4m3", F16, 64, 3, 8, 0, False, False, [1, 1, 1], [9, 8, 100]),
    ("e4m3", BF16, 256, 2, 32, 0, False, False, [1, 1], [64, 65]),
    ("int8", F16, 64, 1, 8, 0, False, False, [5, 0, 17, 1], [5, 9, 40, 3]),
    ("e4m3", BF16, 128, 2, 16, 0, False, False, [30, 2, 16], [30, 18, 31]),
    ("int8", BF16, 256, 1, 64, 0, False, False, [90], [100]),
    ("int8", BF16, 128, 9, 128, 0, False, False, [300, 7], [333, 130]),  # pages with more new rows than a wave holds
    ("e4m3", F16, 256, 1, 1024, 0, False, False, [1500], [2000]),
    ("e4m3", F16, 64, 17, 256, 0, False, False, [260], [270]),           # more pairs than a workgroup takes
    ("e4m3", BF16, 128, 8, 16, 128, True, False, [1, 1, 1], [1, 50, 16]),
    ("int8", BF16, 128, 2, 16, 128, True, False, [40, 3], [44, 600]),
    ("e4m3", F16, 64, 2, 8, 32, True, True, [21], [500]),
    ("int8", F16, 256, 1, 32, 256, False, False, [70], [71]),
    ("e4m3", BF16, 256, 2, 128, 48, True, True, [150], [300]),
    ("int8", F16, 64, 3, 16, 16, False, True, [1, 1], [7, 500000]),
    ("e4m3", BF16, 128, 1, 256, 64, True, False, [700], [800]),
    # two and four waves to a head, pages with rows before the first, more heads than a workgroup takes
    ("e4m3", BF16, 128, 5, 64, 128, True, False, [100, 40, 20], [130, 45, 83]),
    ("int8", F16, 64, 18, 128, 64, True, True, [200, 45], [290, 70]),
    ("int8", BF16, 256, 3, 32, 64, True, False, [31, 12, 50], [40, 12, 60]),
    ("e4m3", F16, 128, 6, 64, 0, False, False, [64, 33], [128, 40]),
    ("int8", BF16, 128, 2, 16, 64, True, False, [9000], [9007]),  # pages enough for all heads together
    ("e4m3", BF16, 64, 33, 32, 64, True, True, [9, 0, 12000], [20, 3, 12011]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(case):
    kind, dtype, D, H, page, R, norm, il, new, lens = case
    s = _batch(sum(new) * 3 + D + page, kind, dtype, D, H, page, new, [min(n, 13000) for n in lens], R, norm, il)
    s["positions"] += max(lens) - min(max(lens), 13000)
    d = _device(s)
    _call(d)
    _compare(s, d, "by offsets")
    once = {x: d[x].clone() for x in ("k_cache", "v_cache", "k_scale", "v_scale")}
    _call(d)  # again: the same rows to the same places
    assert all(torch.equal(d[x].view(torch.uint8) if d[x].dtype != torch.float32 else d[x], once[x].view(torch.uint8)
                           if once[x].dtype != torch.float32 else once[x]) for x in once)
    for more in [dict(max_q_len=max(new))] + ([dict(equal=True)] if len(set(new)) == 1 else []):
        d = _device(s)
        _call(d, **more)
        assert all(torch.equal(d[x], once[x]) for x in once), more


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("pieces", [[1] * 40, [3, 1, 7, 1, 1, 20, 2, 5], [40]], ids=str)
def test_a_page_that_grows(kind, pieces):
    """A request in pieces: after each, codes and scales are what the form makes of those before; at the end every value
    is within the code's own half step of the page's scale, or one step of an int8 code however often the page grew."""
    D, H, page = 64, 2, 16
    s = _batch(4, kind, BF16, D, H, page, [40], [40], spread=9)
    whole = s["kv"]
    for x in "kv":
        s[x + "_scale"].fill_(2.0 ** 40)  # of rows that are no more: a page's first row forgets it
    at = 0
    for n in pieces:
        step = dict(s, kv=whole[at:at + n], kv_len=torch.tensor([at + n], dtype=torch.int32),
                    cu=torch.tensor([0, n], dtype=torch.int32), positions=s["positions"][at:at + n])
        d = _device(step)
        _call(d, max_q_len=n)
        _compare(step, d, at)
        for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
            s[x] = d[x].cpu()
        at += n
    pos = torch.arange(40)
    for x, rows in (("k", whole[:, :H]), ("v", whole[:, H:])):
        p, place = s["table"][0].long()[pos // page], pos % page
        scale = s[x + "_scale"][p].double()[..., None]
        got = do.values(s[x + "_cache"], kind)[p, :, place] * scale
        off, size = (got - rows.double()).abs(), rows.double().abs()
        # e4m3: half a step; below the smallest normal code each of up to 18 growths rounds to half a step of 2^-9, each of
        # twice the unit of the one before: less than a step in all
        most = scale * (1.0 if kind == "int8" else 2.0 ** -9) + (0.0 if kind == "int8" else size * 2.0 ** -4)
        assert (off <= most).all(), x


@pytest.mark.parametrize("one", [True, False])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_magnitudes_and_what_is_not_finite(kind, one):
    """Zeros, the least and largest numbers, magnitudes at a power's border, infinities and NaN, with rows held and without."""
    D, H, page = 64, 2, 8
    for held in (0, 3):
        n = 1 if one else 2
        rows = [0.0, -0.0, 1e-38, 9.2e-41, 3.3e38, 448.0, 450.0, 127.0, 127.5, math.inf, math.nan, -math.inf]
        B = len(rows)
        s = _batch(held + n, kind, BF16, D, H, page, [n] * B, [held + n] * B)
        s["kv"] = torch.zeros((n * B, 2 * H, D), dtype=BF16)
        for i, x in enumerate(rows):
            s["kv"][n * i, 1, 5] = x
            s["kv"][n * i, 2, 63] = x
        for x in "kv":
            s[x + "_scale"][0, 0] = math.nan
            s[x + "_scale"][1] = 0.0
            s[x + "_cache"][1] = 0
        d = _device(s)
        _call(d, max_q_len=n)
        _compare(s, d, held)


def test_what_is_left_out():
    """Requests without keys, tokens before the first key, pages that are none, padding: nothing else changes."""
    for kind, new, lens in (("int8", [1, 1, 1, 1], [0, 5, 20, 7]), ("e4m3", [9, 4, 6, 0], [4, 0, 20, 3])):
        s = _batch(3, kind, BF16, 128, 2, 8, new, [max(n, 0) for n in lens])
        s["positions"] = torch.zeros(sum(new), dtype=torch.int32)
        s["table"][2, 2] = -1                    # the third request's last page
        s["table"][3, 0] = 2 ** 31 - 1
        more = torch.zeros((5, 4, 128), dtype=BF16)  # tokens past the last request
        d = _device(dict(s, kv=torch.cat([s["kv"], more + 100])))
        _call(d)
        _compare(s, d, kind)
        untouched = _device(s)
        empty = dict(untouched, table=untouched["table"][:, :0])  # no pages at all
        _call(empty)
        assert all(torch.equal(empty[x].cpu(), s[x]) for x in ("k_cache", "v_cache", "k_scale", "v_scale"))
    # lengths past the table
    s = _batch(9, "int8", F16, 64, 1, 8, [4], [100])
    s["table"] = s["table"][:, :12].contiguous()  # 96 keys
    d = _device(s)
    _call(d)
    _compare(s, d)


def test_scales_that_are_no_powers_of_two():
    """A scale from elsewhere stays where it is large enough; codes are within a step of its quotients."""
    D, page = 64, 8
    for kind in ("int8", "e4m3"):
        s = _batch(8, kind, BF16, D, 1, page, [1], [4], spread=0)
        for x in "kv":
            s[x + "_scale"].fill_(0.3)
        d = _device(s)
        _call(d)
        p = int(s["table"][0, 0])
        for x, row in (("k", s["kv"][0, 0]), ("v", s["kv"][0, 1])):
            assert (d[x + "_scale"].cpu() == s[x + "_scale"]).all()
            got = do.values(d[x + "_cache"].cpu(), kind)[p, 0, 3] * float(s[x + "_scale"][p, 0])
            size = row.double().abs()
            half = 0.15 if kind == "int8" else size * 2.0 ** -4 + 0.3 * 2.0 ** -10
            assert ((got - row.double()).abs() <= half + 4 * so.U32 * size).all()
            assert torch.equal(d[x + "_cache"].cpu()[:, :, :3], s[x + "_cache"][:, :, :3])


def test_strides_and_halves_of_one_pool():
    """K and V as halves of one allocation, tokens and heads apart, fp8 tensors."""
    D, H, page = 64, 3, 8
    s = _batch(6, "e4m3", BF16, D, H, page, [11], [13])
    want = _device(s)
    _call(want)
    pages = s["k_cache"].shape[0]
    both = torch.zeros((pages, 2, H, page, D), dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = s["k_cache"].cuda(), s["v_cache"].cuda()
    wide = torch.full((11, 2 * H + 1, D + 8), math.nan, dtype=BF16, device="cuda")
    wide[:, :2 * H, :D] = s["kv"].cuda()
    d = _device(s)
    lib().kv_append_pages(wide[:, :H, :D], wide[:, H:2 * H, :D], both[:, 0].view(torch.float8_e4m3fn),
                          both[:, 1].view(torch.float8_e4m3fn), d["k_scale"], d["v_scale"], d["table"], d["kv_len"])
    assert torch.equal(both[:, 0], want["k_cache"]) and torch.equal(both[:, 1], want["v_cache"])
    assert torch.equal(d["k_scale"], want["k_scale"]) and torch.equal(d["v_scale"], want["v_scale"])


def test_replays():
    """A captured append of single tokens and of runs, replayed over growing requests, against eager calls."""
    for n in (1, 3):
        lens = [n] * 3
        s = _batch(12, "int8", BF16, 128, 2, 8, [n] * 3, [40] * 3, 128, True)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32)
        d, e = _device(s), _device(s)
        _call(_device(s), equal=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _call(d, equal=True)
        g = _gen(2)
        for k in range(6):
            new = _normal(tuple(s["kv"].shape), BF16, g, 2.0 ** k)
            for x in (d, e):
                x["kv"].copy_(new)
                x["kv_len"].copy_(torch.tensor([n * (k + 1)] * 3))
                x["positions"].copy_(torch.arange(n * k, n * k + n).repeat(3))
            graph.replay()
            torch.cuda.synchronize()
            _call(e, equal=True)
            assert all(torch.equal(d[x], e[x]) for x in ("k_cache", "v_cache", "k_scale", "v_scale")), (n, k)
