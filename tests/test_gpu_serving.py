"""Head norm + rotation, paged cache append and paged attention against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import serving_oracle as so
from gpu_support import lib

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
# P is held as a 16-bit value and its 16-bit remainder: off by the square of half a step
P_SPLIT = {BF16: 2.0 ** -16, F16: 2.0 ** -20}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(shape, dtype, g, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def _freq(rotary, base=1e4):
    return base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)


def _close(got, want, bound, what):
    got = got.double().cpu()
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off - bound).max()):.3g}"


NORM_ROPE = [
    # tokens, q heads, k heads, dim, rotary, interleaved, weights, dtype, first position
    (1, 32, 8, 128, 128, False, True, BF16, 8191),
    (1, 1, 1, 64, 16, True, True, F16, 0),
    (3, 5, 1, 64, 64, True, False, BF16, 2 ** 31 - 4),
    (17, 14, 2, 64, 32, True, True, F16, 500000),
    (65, 7, 3, 128, 48, False, True, F16, 1000),
    (33, 4, 4, 256, 256, False, True, BF16, 77),
    (9, 3, 2, 256, 0, False, True, BF16, 0),
    (2049, 9, 1, 128, 64, False, True, BF16, 0),  # a wave takes all rows of its token from 2,048 tokens on
    (2048, 2, 2, 256, 128, True, True, F16, 3),
]


@pytest.mark.parametrize("case", NORM_ROPE, ids=str)
def test_norm_rope(case):
    T, Hq, Hk, D, R, il, weights, dtype, first = case
    g = _gen(T * 31 + D)
    qkv = _normal((T, Hq + 2 * Hk, D), dtype, g, 2.0)
    wq, wk = (_normal((D,), dtype, g) + 1 if weights else None for _ in range(2))
    pos = torch.arange(first, first + T, dtype=torch.int64).to(torch.int32)
    freq = _freq(R) if R else None
    d = qkv.cuda()
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    q, k = lib().qk_norm_rope(d[:, :Hq], d[:, Hq:Hq + Hk], dev(pos), dev(freq), q_weight=dev(wq), k_weight=dev(wk),
                              eps=1e-5, interleaved=il)
    for got, x, w, what in ((q, qkv[:, :Hq], wq, "q"), (k, qkv[:, Hq:Hq + Hk], wk, "k")):
        want, fp = so.norm_rope(x, w, 1e-5, pos, freq, il)
        _close(got, want, so.rounding_bound(want, fp, dtype), what)
    assert torch.equal(d.cpu(), qkv)  # the input stays
    # in place, through the strides of the projection's output; one side alone
    lib().qk_norm_rope(None, d[:, Hq:Hq + Hk], dev(pos), dev(freq), k_weight=dev(wk), eps=1e-5, interleaved=il,
                       k_out=d[:, Hq:Hq + Hk])
    assert torch.equal(d[:, Hq:Hq + Hk], k)
    assert torch.equal(d[:, :Hq].cpu(), qkv[:, :Hq]) and torch.equal(d[:, Hq + Hk:].cpu(), qkv[:, Hq + Hk:])


def test_norm_rope_keeps_special_values():
    """A row of zeros stays zero, an infinity or NaN stays in its row; positions below zero turn the other way."""
    x = torch.ones((4, 2, 64), dtype=BF16)
    x[0] = 0
    x[1, 0, 5] = math.inf
    x[2, 1, 63] = math.nan
    pos = torch.tensor([5, -7, 0, -(2 ** 31)], dtype=torch.int32)
    w = torch.full((64,), 0.5, dtype=BF16)
    q, _ = lib().qk_norm_rope(x.cuda(), None, pos.cuda(), _freq(64).cuda(), q_weight=w.cuda())
    q = q.cpu()
    assert (q[0] == 0).all()
    assert q[1, 0].isnan().any() and q[1, 1].isfinite().all()
    assert q[2, 1].isnan().all() and q[2, 0].isfinite().all()
    want, fp = so.norm_rope(x, w, 1e-6, pos, _freq(64), False)
    for t, h in ((1, 1), (2, 0), (3, 0), (3, 1)):
        _close(q[t, h], want[t, h], so.rounding_bound(want[t, h], fp[t, h], BF16), (t, h))


APPEND = [
    # tokens, heads, dim, rotary, interleaved, norm, page, dtype, e4m3
    (1, 1, 64, 0, False, False, 8, BF16, False),
    (1, 8, 128, 128, False, True, 16, BF16, False),
    (67, 3, 128, 64, True, True, 32, F16, False),
    (2050, 2, 256, 256, False, False, 64, BF16, False),
    (1, 8, 128, 128, False, True, 16, BF16, True),
    (131, 5, 64, 48, True, False, 8, F16, True),
    (40, 1, 256, 16, False, True, 1024, F16, True),
    (2061, 4, 128, 128, False, True, 16, BF16, True),
]


def _codes(x):
    """Nearest e4m3 code of each value, by the list of all codes (ties to the even code)."""
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    pos = table[:127]  # 0 .. 448, ascending
    a = x.abs()
    hi = torch.searchsorted(pos, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return pick | (torch.signbit(x).long() << 7)


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case):
    T, H, D, R, il, norm, page, dtype, e4m3 = case
    g = _gen(T + D)
    rng = np.random.default_rng(T)
    qkv = _normal((T, 2 * H + 1, D), dtype, g, 3.0)
    if T > 2:
        qkv[1, 0] = 0
        qkv[2, H] = 0
    k, v = qkv[:, :H], qkv[:, H:2 * H]
    pages = -(-T // page) + 3
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64))
    if T > 10:  # padding and a slot past the pool: nothing is written
        slots[3], slots[7], slots[9] = -1, pages * page, 2 ** 62
    pos = torch.arange(T, dtype=torch.int32) * 977
    freq = _freq(R) if R else None
    w = _normal((D,), dtype, g) + 1 if norm else None
    both = torch.randint(0, 255, (pages, 2, H, page, D * (1 if e4m3 else 2)), generator=g, dtype=torch.uint8)
    if not e4m3:
        both = both.view(dtype)
    scales = torch.rand((2, pages, H, page), generator=g) if e4m3 else None
    c, sc = both.cuda(), None if scales is None else scales.cuda()
    d = qkv.cuda()
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    lib().kv_append(d[:, :H], d[:, H:2 * H], c[:, 0], c[:, 1], dev(slots), positions=dev(pos), inv_freq=dev(freq),
                    k_weight=dev(w), eps=1e-6, interleaved=il, k_scale=None if sc is None else sc[0],
                    v_scale=None if sc is None else sc[1])
    got, got_s = c.cpu(), None if sc is None else sc.cpu()
    keep = (slots >= 0) & (slots < pages * page)
    at_page, at = slots[keep] // page, slots[keep] % page
    k64, fp = so.norm_rope(k, w, 1e-6, pos, freq, il)
    for side, want, fp in ((0, k64[keep], fp[keep]), (1, v[keep].double(), torch.zeros_like(fp[keep]))):
        rows = got[:, side][at_page, :, at]
        if not e4m3:
            if side == 1:
                assert torch.equal(rows, v[keep])
            else:
                _close(rows, want, so.rounding_bound(want, fp, dtype), "k")
            continue
        scale = got_s[side][at_page, :, at].double()
        amax = want.abs().amax(-1)
        assert ((scale - amax / 448).abs() <= (fp.amax(-1) + 2 * so.U32 * amax) / 448).all()
        quotient = torch.where(amax[..., None] > 0, want * 448 / amax[..., None], 0.0 * want)
        code = rows.view(torch.float8_e4m3fn).double()
        if side == 1:
            assert torch.equal(rows.long(), _codes(quotient))
        # half a step (steps of 2^-9 below 2^-6) of the quotient, and what fp32 moved it by
        moved = torch.where(amax[..., None] > 0, (fp + fp.amax(-1, keepdim=True)) * 448 / amax[..., None], 0.0 * want)
        bound = (quotient.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 8 * so.U32) + 2 * moved
        _close(code, quotient, bound, ("codes", side))
    # what was not named keeps its bits
    named = torch.zeros(pages * page, dtype=torch.bool)
    named[slots[keep]] = True
    rest = (~named).reshape(pages, page)
    for side in (0, 1):
        bits = [x[:, side].transpose(1, 2)[rest].contiguous().view(torch.uint8) for x in (got, both)]
        assert torch.equal(*bits)
        if e4m3:
            assert torch.equal(got_s[side].transpose(1, 2)[rest], scales[side].transpose(1, 2)[rest])


def test_append_special_rows():
    """NaN and infinity reach the row's scale; huge and tiny rows keep their codes; nothing spills over."""
    T, D, page = 6, 64, 8
    x = torch.ones((T, 1, D), dtype=BF16)
    x[0, 0, 3] = math.nan
    x[1, 0, 4] = -math.inf
    x[2] = 3e38
    x[2, 0, 1] = -1.5e38
    x[3] = 1e-38
    x[4] = 0
    c = [torch.zeros((1, 1, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.zeros((1, 1, page), device="cuda") for _ in range(2)]
    lib().kv_append(x.cuda(), x.cuda(), c[0], c[1], torch.arange(T).cuda(), k_scale=s[0], v_scale=s[1])
    for cache, scale in zip(c, s):
        value = cache.cpu().view(torch.float8_e4m3fn).double()[0, 0]
        scale = scale.cpu().double()[0, 0]
        assert scale[0].isnan() and scale[1].isinf()
        assert (value[0] * scale[0]).isnan().all() and (value[1] * scale[1])[4].isnan()
        for t in (2, 3, 5):
            assert (value[t] * scale[t] - x[t, 0].double()).abs().max() <= x[t, 0].double().abs().max() * 2.0 ** -4
        assert (value[2, 0], value[2, 1]) == (448, -224) and (value[3] == 448).all()
        assert (value[4] == 0).all() and scale[4] == 0
        assert (value[6:] == 0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _paged(seed, dtype, e4m3, D, H, G, page, q_lens, kv_lens, spare=2, extra=0, equal=False):
    """A pool of pages in random order, with NaN in every place that no request holds."""
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    B = len(q_lens)
    need = [-(-max(n, 0) // page) for n in kv_lens]
    width = max(need + [1]) + extra
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((B, width), 2 ** 30, dtype=np.int32)  # entries past a request's pages are no pages
    used = np.zeros((pages, page), dtype=bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        for i in range(n):
            used[order[at + i], :max(0, min(page, kv_lens[b] - i * page))] = True
        at += n
    used = torch.from_numpy(used)
    s = {"D": D, "H": H, "G": G, "page": page, "dtype": dtype,
         "q": _normal((sum(q_lens), H * G, D), dtype, g, 1.5),
         "table": torch.from_numpy(table), "kv_len": torch.tensor(kv_lens, dtype=torch.int32),
         "cu": torch.from_numpy(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)),
         "equal": equal, "k_scale": None, "v_scale": None}
    for x in "kv":
        r = torch.randn((pages, H, page, D), generator=g)
        if e4m3:
            scale = r.abs().amax(-1) / 448
            codes = (r / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            codes.transpose(1, 2)[~used] = 0x7F
            scale.transpose(1, 2)[~used] = math.nan
            s[x], s[x + "_scale"] = codes, scale
        else:
            r = r.to(dtype)
            r.transpose(1, 2)[~used] = math.nan
            s[x] = r
    return s


def _attend(s, window=0, scale=None, lse=True, **more):
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    return lib().paged_attention(c(s["q"]), c(s["k"]), c(s["v"]), c(s["table"]), c(s["kv_len"]),
                                 cu_q=None if s["equal"] else c(s["cu"]), scale=scale, window=window,
                                 k_scale=c(s["k_scale"]), v_scale=c(s["v_scale"]), return_lse=lse, **more)


def _p_half_step(s, max_rows):
    return P_SPLIT[BF16 if s["k_scale"] is not None else s["dtype"]]


def _compare(s, got, window=0, scale=None, max_rows=16):
    scale = s["D"] ** -0.5 if scale is None else scale
    out, lse, mass, move = so.attention(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["cu"], scale, window,
                                        s["k_scale"], s["v_scale"])
    ob, lb = so.attention_bounds(out, lse, mass, move, s["dtype"], _p_half_step(s, max_rows))
    _close(got[0], out, ob, "out")
    l = got[1].double().cpu()
    empty = lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert (got[0].cpu()[empty] == 0).all()
    _close(torch.where(empty, 0.0, l), torch.where(empty, 0.0, lse), torch.where(empty, 0.0, lb), "lse")


DECODE = [
    # dtype, e4m3, dim, kv heads, group, page, window, kv lengths
    (BF16, False, 128, 1, 1, 16, 0, [1]),
    (BF16, False, 128, 8, 4, 16, 0, [512]),
    (BF16, False, 128, 2, 4, 16, 0, [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]),
    (F16, False, 64, 2, 7, 8, 0, [5, 1000, 77]),
    (F16, False, 256, 1, 5, 32, 0, [999, 64]),
    (BF16, False, 64, 3, 16, 128, 0, [130, 1]),
    (BF16, False, 128, 1, 17, 64, 0, [100]),       # a group over one tile's rows
    (BF16, False, 128, 2, 2, 16, 1, [40, 1, 0]),   # a window of one key
    (F16, False, 128, 2, 3, 16, 100, [50, 100, 101, 5000]),
    (BF16, False, 128, 1, 2, 8, 0, [9001]),        # more than 1,024 pages in a split's range; many splits
    (BF16, True, 128, 8, 4, 32, 0, [700, 3, 64]),
    (F16, True, 64, 2, 8, 16, 0, [1, 4097]),
    (F16, True, 256, 1, 3, 8, 33, [200, 10]),
    (BF16, True, 256, 2, 1, 1024, 0, [1500]),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_attention_single_tokens(case):
    dtype, e4m3, D, H, G, page, window, lens = case
    s = _paged(len(lens) * 7 + D + page, dtype, e4m3, D, H, G, page, [1] * len(lens), lens, equal=True)
    got = _attend(s, window)
    _compare(s, got, window)
    again = _attend(s, window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])  # the same bits on every call
    s["equal"] = False  # the same batch by its offsets
    ragged = _attend(s, window, max_q_len=1)
    assert torch.equal(got[0], ragged[0]) and torch.equal(got[1], ragged[1])


RUNS = [
    # dtype, e4m3, dim, kv heads, group, page, window, new tokens, kv lengths
    (BF16, False, 128, 2, 4, 16, 0, [3, 0, 1, 4, 0], [3, 9, 0, 2, 0]),  # rows before the first key, requests of none
    (F16, False, 64, 1, 1, 8, 0, [16, 5], [700, 5]),
    (BF16, False, 64, 2, 3, 16, 7, [5, 2], [50, 6]),
    (BF16, True, 128, 2, 2, 16, 0, [6, 1, 8], [300, 40, 8]),
    (F16, True, 64, 1, 4, 32, 20, [4, 3], [1000, 33]),
]


@pytest.mark.parametrize("case", RUNS, ids=str)
def test_attention_short_runs(case):
    dtype, e4m3, D, H, G, page, window, new, lens = case
    s = _paged(sum(new) + D, dtype, e4m3, D, H, G, page, new, lens, extra=2)
    got = _attend(s, window, max_q_len=max(new))
    _compare(s, got, window)


def test_attention_many_requests_by_offsets():
    """Requests beyond one step of the search for a tile's request, empty ones among them."""
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 4, 300)]
    lens = [int(rng.integers(n, 60)) for n in new]
    s = _paged(11, BF16, False, 64, 1, 3, 8, new, lens)
    _compare(s, _attend(s, max_q_len=3))


def test_attention_hides_what_is_masked():
    """NaN and infinities in keys and values that a token may not see change nothing."""
    new, lens = [5, 2], [37, 12]
    for e4m3 in (False, True):
        s = _paged(5, BF16, e4m3, 128, 1, 2, 8, new, lens)
        clean = _attend(s)
        page, at = int(s["table"][0, 36 // 8]), 36 % 8  # the last token's own key and value
        if e4m3:
            s["k"][page, 0, at, 3] = 0x7F
            s["v"][page, 0, at, 9] = 0xFF
        else:
            s["k"][page, 0, at, 3] = math.inf
            s["v"][page, 0, at, 9] = -math.inf
            s["v"][page, 0, at, 70] = math.nan
        out, lse = _attend(s)
        assert torch.equal(out[:4], clean[0][:4]) or (out[:4].float() - clean[0][:4].float()).abs().max() <= 2 ** -8 * 4
        assert out[:4].isfinite().all() and lse[:4].isfinite().all()
        assert out[4].isnan().any()
        assert torch.equal(out[5:], clean[0][5:])
        # a window hides the oldest keys in the same way
        s = _paged(6, BF16, e4m3, 64, 1, 1, 8, [3], [40])
        page = int(s["table"][0, 0])
        if e4m3:
            s["v_scale"][page, 0, 0:2] = math.nan
        else:
            s["v"][page, 0, 0:2] = math.nan
        out, _ = _attend(s, window=37)  # tokens 37, 38, 39 see keys from 1, 2, 3 on
        assert out[0].isnan().any() and out[1:].isfinite().all()
        fixed = dict(s)
        fixed["q"], fixed["cu"] = s["q"][1:], torch.tensor([0, 2], dtype=torch.int32)
        _compare(fixed, _attend(fixed, window=37), window=37)


def test_attention_skips_pages_outside_the_pool():
    s = _paged(9, F16, False, 64, 2, 2, 8, [1, 1, 1], [50, 20, 8], equal=True)
    s["table"][0, 2] = -1
    s["table"][0, 4] = 2 ** 31 - 1
    s["table"][2, 0] = -5  # its only page: a row without keys
    got = _attend(s)
    _compare(s, got)
    assert (got[0][2] == 0).all() and (got[1][2] == -math.inf).all()


def test_attention_bounds_lengths():
    """Lengths below zero and past the table are bounded by what the table holds."""
    s = _paged(10, BF16, False, 64, 1, 2, 8, [1, 1], [16, 16], equal=True)
    s["kv_len"] = torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32)
    _compare(s, _attend(s))


def test_attention_extreme_scores():
    """Scores far apart, all equal, and very negative: the running maximum carries them."""
    s = _paged(12, F16, False, 64, 1, 4, 16, [1, 1], [600, 33], equal=True)
    for scale in (0.0, 20.0, -20.0, 1e-6):
        _compare(s, _attend(s, scale=scale), scale=scale)
    s["k"][~s["k"].isnan()] = 30000.0
    s["q"][:] = -60.0
    got = _attend(s, scale=1.0)
    assert got[0].isfinite().all() and got[1].isfinite().all()


def test_attention_strided_and_out():
    """Slices of one projection's output, a cache of halves of one allocation, a table with wider rows, given outputs."""
    s = _paged(13, BF16, False, 128, 2, 2, 16, [2, 3], [40, 50])
    plain = _attend(s)
    T = 5
    packed = torch.zeros((T, 9, 128), dtype=BF16, device="cuda")
    packed[:, 2:6] = s["q"].cuda()
    both = torch.stack([s["k"], s["v"]], 1).cuda()
    wide = torch.full((2, s["table"].shape[1] + 5), -1, dtype=torch.int32)
    wide[:, :s["table"].shape[1]] = s["table"]
    wide = wide.cuda()
    out = torch.full((T, 6, 128), 7.0, dtype=BF16, device="cuda")
    got = lib().paged_attention(packed[:, 2:6], both[:, 0], both[:, 1], wide[:, :s["table"].shape[1]],
                                s["kv_len"].cuda(), cu_q=s["cu"].cuda(), out=out[:, 1:5])
    assert torch.equal(got, plain[0]) and (out[:, 0] == 7).all() and (out[:, 5] == 7).all()


def test_attention_on_another_stream_with_its_workspace():
    s = _paged(14, BF16, False, 128, 1, 4, 16, [1], [5000], equal=True)
    here = _attend(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = _attend(s, stream=side)
        side.synchronize()
        assert torch.equal(got[0], here[0])
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    assert torch.equal(_attend(s, workspace=ws)[0], here[0])


def test_a_step_in_a_graph():
    """Norm, append and attention of a decode step, captured and replayed over changing inputs, against eager runs."""
    hg = lib()
    B, H, G, D, page = 5, 2, 4, 64, 16
    g = _gen(21)
    lens = [3, 17, 64, 1000, 2500]
    s = _paged(21, BF16, False, D, H, G, page, [1] * B, lens, equal=True)
    kc, vc, table = s["k"].cuda(), s["v"].cuda(), s["table"].cuda()
    freq, w = _freq(D).cuda(), (_normal((D,), BF16, g) + 1).cuda()
    x = torch.zeros((B, H * G + 2 * H, D), dtype=BF16, device="cuda")
    pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    slots = torch.tensor([int(s["table"][b, (n - 1) // page]) * page + (n - 1) % page for b, n in enumerate(lens)]).cuda()
    kv_len = s["kv_len"].cuda()

    def step(ws=None):
        q, _ = hg.qk_norm_rope(x[:, :H * G], None, pos, freq, q_weight=w)
        hg.kv_append(x[:, H * G:H * G + H], x[:, H * G + H:], kc, vc, slots, positions=pos, inv_freq=freq, k_weight=w)
        return hg.paged_attention(q, kc, vc, table, kv_len)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_normal(tuple(x.shape), BF16, g))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())


def test_binding_refuses():
    """Shapes, types and layouts that the binding refuses; nothing is launched."""
    hg = lib()
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    q, k, cache, slots = z(2, 8, 64), z(2, 2, 64), z(4, 2, 16, 64), z(2, t=torch.int64)
    pos, freq, table, lens = z(2, t=torch.int32), z(32, t=torch.float64), z(2, 2, t=torch.int32), z(2, t=torch.int32)
    codes, scale = z(4, 2, 16, 64, t=torch.uint8), z(4, 2, 16, t=torch.float32)
    bad = [
        lambda: hg.qk_norm_rope(q, k[:1]), lambda: hg.qk_norm_rope(q, k.half()), lambda: hg.qk_norm_rope(q, z(2, 2, 128)),
        lambda: hg.qk_norm_rope(q, k, None, freq),
        lambda: hg.qk_norm_rope(q, k, pos, freq.float()), lambda: hg.qk_norm_rope(q, k, pos.long(), freq),
        lambda: hg.qk_norm_rope(q, k, pos[:1], freq), lambda: hg.qk_norm_rope(q, k, q_weight=z(32)),
        lambda: hg.qk_norm_rope(q.transpose(1, 2), None), lambda: hg.qk_norm_rope(q, None, k_weight=z(64)),
        lambda: hg.qk_norm_rope(q, None, q_out=z(2, 8, 64).half()), lambda: hg.qk_norm_rope(q, None, q_out=z(3, 8, 64)),
        lambda: hg.qk_norm_rope(q, None, q_out=z(1, 8, 64).expand(2, 8, 64)), lambda: hg.qk_norm_rope(q[0], None),
        lambda: hg.qk_norm_rope(q.clone().requires_grad_(), None),
        lambda: hg.kv_append(q, q, cache, cache, slots), lambda: hg.kv_append(k, k[:1], cache, cache, slots),
        lambda: hg.kv_append(k, k, cache, cache[:2], slots), lambda: hg.kv_append(k, k, cache.half(), cache.half(), slots),
        lambda: hg.kv_append(k, k, cache, cache, slots.int()), lambda: hg.kv_append(k, k, cache, cache, slots[:1]),
        lambda: hg.kv_append(k, k, codes, codes, slots), lambda: hg.kv_append(k, k, cache, cache, slots, k_scale=scale),
        lambda: hg.kv_append(k, k, codes, codes, slots, k_scale=scale, v_scale=scale.double()),
        lambda: hg.kv_append(k, k, cache.transpose(1, 2), cache.transpose(1, 2), slots),
        lambda: hg.paged_attention(q, cache, cache, table.long(), lens),
        lambda: hg.paged_attention(q, cache, cache, table, lens[:1]), lambda: hg.paged_attention(q, cache, cache, table.T, lens),
        lambda: hg.paged_attention(q, cache, cache, table, lens, cu_q=lens),
        lambda: hg.paged_attention(q, cache, cache, table, lens, out=q.half()),
        lambda: hg.paged_attention(q, cache, cache, table, lens, workspace=scale),
        lambda: hg.paged_attention(q, cache.float(), cache.float(), table, lens),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, hg.EngramError)):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: hg.paged_attention(z(2, 7, 64), cache, cache, table, lens),
                 lambda: hg.paged_attention(q, cache, cache, table, lens, scale=math.nan),
                 lambda: hg.paged_attention(q, cache, cache, table, lens, window=-1),
                 lambda: hg.kv_append(z(2, 2, 96), z(2, 2, 96), z(4, 2, 16, 96), z(4, 2, 16, 96), slots),
                 lambda: hg.qk_norm_rope(z(2, 8, 68)[..., 2:66], None)):
        with pytest.raises(hg.EngramError):
            call()


def test_of_nothing():
    hg = lib()
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    i = torch.int32
    cache = z(4, 2, 16, 64)
    q, k = hg.qk_norm_rope(z(0, 8, 64), z(0, 2, 64), z(0, t=i), z(32, t=torch.float64))
    assert q.shape == (0, 8, 64) and k.shape == (0, 2, 64)
    hg.kv_append(z(0, 2, 64), z(0, 2, 64), cache, cache, z(0, t=torch.int64))
    assert hg.paged_attention(z(0, 8, 64), cache, cache, z(0, 2, t=i), z(0, t=i)).shape == (0, 8, 64)
    # requests without tokens, and tokens without a page
    assert hg.paged_attention(z(0, 8, 64), cache, cache, z(3, 2, t=i), z(3, t=i), cu_q=z(4, t=i)).shape == (0, 8, 64)
    out, lse = hg.paged_attention(z(2, 8, 64) + 1, cache, cache, z(2, 0, t=i), z(2, t=i) + 5, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
