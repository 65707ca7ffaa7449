"""A cache whose pages lie past 2^32 elements: the same bits as from a small one."""
import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_past_32_bits(e4m3):
    hg = lib()
    page, D, G, n = 1024, 128, 4, 2500
    many = 17000  # K and V in one allocation: 2^18 elements from page to page
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn((n, 1, D), generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn((60, G, D), generator=g).to(BF16).cuda()
    got = []
    for pages, ids in ((3, [0, 1, 2]), (many, [many - 1, 16390, many - 2])):
        both = torch.empty((pages, 2, 1, page, D), dtype=torch.uint8 if e4m3 else BF16, device="cuda")
        scales = [torch.empty((pages, 1, page), device="cuda") for _ in range(2)] if e4m3 else [None, None]
        at = torch.arange(n)
        slots = (torch.tensor(ids)[at // page] * page + at % page).cuda()
        hg.kv_append(k, v, both[:, 0], both[:, 1], slots, k_scale=scales[0], v_scale=scales[1])
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        for new in (1, 60):
            got.append(hg.paged_attention(q[:new], both[:, 0], both[:, 1], table, lens, k_scale=scales[0], v_scale=scales[1]))
        torch.cuda.synchronize()
        del both
    torch.cuda.empty_cache()
    assert got[0].isfinite().all() and got[1].isfinite().all()
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
