"""Pages and scales past 2^32 elements, each operator by itself: what it reads or writes is placed by torch's indexing."""
import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16, F16

pytestmark = pytest.mark.gpu

PAGE, H, D, N = 1024, 2, 64, 2500
STRIDE = 2 * H * PAGE * D  # elements from page to page: K and V are halves of one allocation
MANY = 2 ** 32 // STRIDE + 500


def _ids():
    """Pages past 2^32 elements, and where their offsets would land in 32 bits: all apart, all in the pool."""
    far = [MANY - 1, MANY - 300, MANY - 2]
    near = [i * STRIDE % 2 ** 32 // STRIDE for i in far]
    assert all(i * STRIDE >= 2 ** 32 for i in far) and len({*far, *near}) == 6
    return far, near


def _rows(dtype, e4m3, seed):
    x = torch.randn((2, N, H, D), generator=torch.Generator().manual_seed(seed)).to(dtype)
    if not e4m3:
        return x, None
    s = x.float().abs().amax(-1) / 448
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _pool(dtype, e4m3):
    both = torch.empty((MANY, 2, H, PAGE, D), dtype=torch.uint8 if e4m3 else dtype, device="cuda")
    assert both.stride(0) == STRIDE
    return both


@pytest.mark.parametrize("dtype,e4m3", [(BF16, False), (F16, True)], ids=str)
def test_append_writes_far_pages(dtype, e4m3):
    far, near = _ids()
    x = torch.randn((2, N, H, D), generator=torch.Generator().manual_seed(5)).to(dtype)
    both = _pool(dtype, e4m3)
    scales = torch.empty((2, MANY, H, PAGE), device="cuda") if e4m3 else [None, None]
    mark = 0x41 if e4m3 else 7.0
    both[far + near] = mark
    at = torch.arange(N)
    page, place = torch.tensor(far)[at // PAGE], at % PAGE
    k, v = x.cuda()
    lib().kv_append(k, v, both[:, 0], both[:, 1], (page * PAGE + place).cuda(), k_scale=scales[0], v_scale=scales[1])
    assert (both[near] == mark).all()
    for side in range(2):
        rows = both[page.cuda(), side, :, place.cuda()].cpu()
        if not e4m3:
            assert torch.equal(rows, x[side])
            continue
        s = scales[side][page.cuda(), :, place.cuda()].cpu()
        amax = x[side].double().abs().amax(-1)
        assert ((s.double() * 448 - amax).abs() <= 2.0 ** -22 * amax).all()
        # half a step of the code, 2^-4 of it and 2^-10 of the scale at least
        off = (rows.view(torch.float8_e4m3fn).double() * s.double()[..., None] - x[side].double()).abs()
        assert (off <= 1.001 * (x[side].double().abs() * 2.0 ** -4).clamp(min=amax[..., None] * 2.0 ** -10 / 448)).all()
    left = both[far[2], :, :, N % PAGE:]
    assert (left == mark).all()


@pytest.mark.parametrize("dtype,e4m3", [(BF16, False), (F16, True)], ids=str)
@pytest.mark.parametrize("new", [1, 80])
def test_attention_reads_far_pages(dtype, e4m3, new):
    """The bits of a small pool with the same rows; NaN in the places that 32 bits would lead to."""
    far, near = _ids()
    codes, s = _rows(dtype, e4m3, 6)
    q = torch.randn((new, 4 * H, D), generator=torch.Generator().manual_seed(new)).to(dtype).cuda()
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    at = torch.arange(N)
    got = []
    for ids, bad in (([0, 1, 2], []), (far, near)):
        both = _pool(dtype, e4m3) if bad else torch.empty((3, 2, H, PAGE, D), dtype=codes.dtype, device="cuda")
        scales = torch.empty((2, both.shape[0], H, PAGE), device="cuda") if e4m3 else [None, None]
        both[ids + bad] = 0x7F if e4m3 else float("nan")
        page, place = torch.tensor(ids)[at // PAGE].cuda(), (at % PAGE).cuda()
        for side in range(2):
            both[page, side, :, place] = codes[side].cuda()
            if e4m3:
                scales[side][ids + bad] = float("nan")
                scales[side][page, :, place] = s[side].cuda()
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        got.append(lib().paged_attention(q, both[:, 0], both[:, 1], table, lens, k_scale=scales[0], v_scale=scales[1]))
    assert got[0].isfinite().all()
    assert torch.equal(got[0], got[1])
