"""Requests of as many keys as there can be: a window near 2^31 gives the bits of one near 0."""
import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16

pytestmark = pytest.mark.gpu

PAGE = 1024


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,D", [(1, 64), (3, 128), (50, 64), (300, 128), (40, 256)])
@pytest.mark.parametrize("back", [0, 1000])
def test_windows_at_the_longest_request(e4m3, new, D, back):
    H, G, window, width = 1, 2, 500, 1 << 21  # 2^31 places
    g = torch.Generator().manual_seed(new + D)
    x = torch.randn((2, 2, H, PAGE, D), generator=g)
    scales = [None, None]
    if e4m3:
        s = x.abs().amax(-1) / 448
        scales, x = list(s.cuda()), (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = x.to(BF16)
    k, v = x.cuda()
    q = torch.randn((new, H * G, D), generator=g).to(BF16).cuda()
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    longest = 2 ** 31 - 4096
    got = []
    # the window lies on two pages whose first keys are multiples of 1,024 in both
    for length in (longest - back, 8 * PAGE - back):
        table.fill_(-1)
        last = (length - 1) // PAGE
        table[0, last - 1], table[0, last] = (1, 0) if last % 2 else (0, 1)
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        got.append(lib().paged_attention(q, k, v, table, lens, window=window, k_scale=scales[0], v_scale=scales[1], return_lse=True))
    assert got[0][0].isfinite().all() and got[0][1].isfinite().all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    if back == 0:  # lengths past the longest are bounded by it
        last = (longest - 1) // PAGE
        table.fill_(-1)
        table[0, last - 1], table[0, last] = (1, 0) if last % 2 else (0, 1)
        lens.fill_(2 ** 31 - 1)
        again = lib().paged_attention(q, k, v, table, lens, window=window, k_scale=scales[0], v_scale=scales[1])
        assert torch.equal(again, got[0][0])
