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


def _by_declaration(s, sides=(("k", slice(0, 2)), ("v", slice(2, 4)))):
    """One request's rows, as given, appended in 64 bits: {side: (values of the codes, scales)} of its pages."""
    found, (length, n, page) = {}, (int(s["kv_len"][0]), s["kv"].shape[0], s["k_cache"].shape[2])
    for x, cols in sides:
        value, scale = do.values(s[x + "_cache"], s["kind"]), s[x + "_scale"].double().clone()
        for key0 in range((length - n) // page * page, length, page):
            p, a, e = int(s["table"][0, key0 // page]), max(length - n, key0), min(length, key0 + page)
            rows = s["kv"][a - (length - n):e - (length - n), cols].transpose(0, 1).double()  # [H, n, D]
            need = do.power_of_two(rows.abs().amax((1, 2)) / do.LARGEST[s["kind"]])
            old = scale[p].clone()
            more = (need > old.abs()) if a > key0 else torch.ones(2, dtype=torch.bool)
            scale[p] = torch.where(more, need, old)
            held = value[p, :, :a - key0]
            if s["kind"] == "int8":
                held = torch.where((old < 0)[:, None, None] & more[:, None, None], held.clamp(min=-127), held)
            value[p, :, :a - key0] = torch.where(more[:, None, None], do.nearest(held * (old / scale[p])[:, None, None], s["kind"]),
                                                 held)
            value[p, :, a - key0:e - key0] = do.nearest(rows / scale[p][:, None, None], s["kind"])
        found[x] = value, scale
    return found


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("new,length,page", [(1, 6, 8), (5, 14, 16), (40, 70, 64), (90, 131, 128)])
def test_scales_below_zero(kind, new, length, page):
    """Negative scales held, larger and smaller in magnitude than the new rows need: codes stay those of their values."""
    for held in (-4.0, -2.0 ** -12, -2.0 ** -5, 0.0, -0.0, 8.0):
        s = _batch(new, kind, BF16, 64, 2, page, [new], [length], spread=1)
        for x in "kv":
            s[x + "_scale"].fill_(held)
            if kind == "int8":
                s[x + "_cache"][:, :, 0, :4] = -128
        d = _device(s)
        _call(d)
        for x, (value, scale) in _by_declaration(s).items():
            assert torch.equal(d[x + "_scale"].cpu().double(), scale), (held, x)
            pages = s["table"][0, :-(-length // page)].long()
            got = do.values(d[x + "_cache"].cpu(), kind)
            assert torch.equal(got[pages], value[pages]), (held, x)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_scale_below_zero_next_to_the_one_that_follows(kind):
    """Held codes times a ratio next to -1, -128 among them, do not leave the codes."""
    new, length, page = 1, 6, 8
    s = _batch(2, kind, BF16, 64, 2, page, [new], [length], spread=0)
    s["kv"][0, :, 0] = 127.0
    s["kv"][0, :, 1:] = 1.0
    need = 1.0 if kind == "int8" else 0.5  # 127 <= need * largest code
    for x in "kv":
        s[x + "_scale"].fill_(-need * (1 - 2.0 ** -20))
        if kind == "int8":
            s[x + "_cache"][:, :, 0] = -128
            s[x + "_cache"][:, :, 1] = 127
    d = _device(s)
    _call(d)
    for x, (value, scale) in _by_declaration(s).items():
        p = int(s["table"][0, 0])
        assert (d[x + "_scale"].cpu()[p] == need).all()
        assert torch.equal(do.values(d[x + "_cache"].cpu(), kind)[p, :, :length], value[p, :, :length])
