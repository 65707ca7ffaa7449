"""Sliding windows whose pages behind them are freed: -1 in the table, and nothing changes."""
import pytest
import torch

from test_gpu_serving import BF16, F16, _attend, _paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,e4m3,D,page,new,lens,window", [
    (BF16, False, 128, 8, [70, 300], [1000, 420], 90),
    (BF16, False, 64, 16, [130], [2100], 333),
    (F16, False, 256, 32, [50, 1], [700, 700], 100),
    (F16, True, 128, 8, [90, 3, 40], [801, 300, 40], 77),
    (BF16, True, 64, 8, [1, 2], [3000, 2000], 1001),  # few rows
], ids=str)
def test_pages_behind_the_window(dtype, e4m3, D, page, new, lens, window):
    s = _paged(sum(lens) + D, dtype, e4m3, D, 2, 2, page, new, lens)
    want = _attend(s, window, max_q_len=max(new))
    assert want[0].isfinite().all()
    freed = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        behind = max(length - n - window + 1, 0) // page  # the first token of the call sees no key of these
        s["table"][b, :behind] = -1
        freed += behind
    assert freed
    got = _attend(s, window, max_q_len=max(new))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
