"""Paged attention of few rows per request where the keys of all requests are shared out between workgroups."""
import math

import numpy as np
import pytest
import torch

from test_gpu_serving import BF16, F16, _attend, _compare, _paged

pytestmark = pytest.mark.gpu


SHARED = [
    # dtype, e4m3, dim, kv heads, group, page, window, new tokens, kv lengths
    (BF16, False, 64, 1, 2, 8, 0, [1], [20000]),                               # one tile over many shares
    (BF16, False, 128, 1, 4, 16, 0, [8, 1, 0, 5], [700, 0, 5, 3000]),          # two tiles; requests of nothing between
    (F16, False, 64, 2, 1, 16, 0, [1] * 5, [4097, 1, 128, 129, 2048]),         # lengths around a block
    (BF16, True, 128, 1, 3, 32, 0, [2, 1, 1], [2500, 640, 1]),
    (F16, True, 64, 1, 8, 8, 700, [1, 3], [5000, 900]),
    (BF16, False, 256, 1, 2, 64, 0, [1, 1], [1500, 300]),
    (BF16, False, 64, 1, 4, 16, 600, [8, 7], [3000, 610]),                   # windows that begin apart within a tile
    (BF16, False, 64, 1, 1, 16, 0, [1, 1], [0, 0]),                            # room for many keys, none there
]


@pytest.mark.parametrize("case", SHARED, ids=str)
def test_shared_keys(case):
    dtype, e4m3, D, H, G, page, window, new, lens = case
    s = _paged(sum(lens) + D, dtype, e4m3, D, H, G, page, new, lens, extra=0 if max(lens) else 100)
    got = _attend(s, window, max_q_len=max(new))
    _compare(s, got, window)
    again = _attend(s, window, max_q_len=max(new))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("n", [64, 65, 300], ids=str)
def test_shared_keys_of_many_requests(n):
    """Up to 64 requests a wave finds its share by itself, beyond by way of LDS; empty requests and lengths among them."""
    rng = np.random.default_rng(n)
    new = [int(rng.choice([0, 1, 1, 2])) for _ in range(n)]
    lens = [int(rng.choice([0, 1, 100, int(rng.integers(1, 1400))])) for _ in range(n)]
    lens[n // 2], new[n // 2] = 1400, 1
    s = _paged(n, BF16, False, 64, 1, 2, 8, new, lens)
    _compare(s, _attend(s, max_q_len=2))


def test_shared_keys_hide_what_is_masked():
    """As for keys that are not shared: NaN and infinities that a token may not see change nothing."""
    n, length = 12, 900
    s = _paged(5, BF16, False, 64, 1, 2, 8, [n], [length])
    clean = _attend(s, max_q_len=n)
    _compare(s, clean)
    at = 895  # seen by the tokens 7 and later
    page, place = int(s["table"][0, at // 8]), at % 8
    s["v"][page, 0, place, 9] = -math.inf
    s["v"][page, 0, place, 40] = math.nan
    out, lse = _attend(s, max_q_len=n)
    assert torch.equal(lse, clean[1])
    assert (out[7:, :, 9] == -math.inf).all() and out[7:, :, 40].isnan().all()
    hidden = dict(s, q=s["q"][:7], cu=torch.tensor([0, 7], dtype=torch.int32), kv_len=torch.tensor([895], dtype=torch.int32))
    _compare(hidden, (out[:7], lse[:7]))
    rest = torch.ones(64, dtype=torch.bool)
    rest[[9, 40]] = False
    assert (out[7:, :, rest].float() - clean[0][7:, :, rest].float()).abs().max() <= 2 ** -7


def test_shared_keys_with_missing_pages_and_wild_lengths():
    s = _paged(9, F16, False, 64, 1, 2, 8, [1, 1, 1], [1400, 900, 700], equal=True)
    s["table"][0, 3] = -1
    s["table"][0, 100] = 2 ** 31 - 1
    s["table"][1] = 2 ** 30
    got = _attend(s)
    _compare(s, got)
    assert (got[0][1] == 0).all() and (got[1][1] == -math.inf).all()
    s = _paged(10, BF16, False, 64, 1, 2, 8, [1, 1], [1000, 1000], equal=True)
    s["kv_len"] = torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32)
    _compare(s, _attend(s))


def test_the_workspace_that_is_asked_for():
    import hashed_gram_memory_amd as hg
    s = _paged(14, BF16, False, 128, 1, 4, 16, [1, 1], [5000, 100], equal=True)
    here = _attend(s)
    args = [s[k].cuda() for k in ("q", "k", "v", "table", "kv_len")]
    need = hg.paged_attention_workspace(*args)
    assert need > 0 and need % 256 == 0
    ws = torch.randint(0, 255, (need,), dtype=torch.uint8, device="cuda")  # what it holds does not matter
    got = hg.paged_attention(*args, return_lse=True, workspace=ws)
    assert torch.equal(got[0], here[0]) and torch.equal(got[1], here[1])
    with pytest.raises(hg.EngramError):
        hg.paged_attention(*args, workspace=ws[:need - 256])
    small = hg.paged_attention_workspace(args[0], args[1], args[2], args[3][:, :4].contiguous(), args[4])
    assert small == 0
