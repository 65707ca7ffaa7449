"""Cosines and sines of the rotation: the fp32 numbers nearest to those of the fp64 angle, at any position."""
import pytest
import torch

from gpu_support import lib
from test_gpu_serving import BF16, F16, _freq

pytestmark = pytest.mark.gpu


def _positions(first):
    g = torch.Generator().manual_seed(3)
    if first is None:  # any int32
        pos = torch.randint(-2 ** 31, 2 ** 31, (16384,), generator=g)
        pos[:3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0])
        return pos.to(torch.int32)
    return torch.arange(first, first + 16384, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("first", [0, 500000, None], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_unit_rows(dtype, first, interleaved):
    """The pair (1, 0) comes back as (cos t, sin t).  Roundings keep the order of numbers, so that a cosine in fp64 within
    2^-30 of the true one, rounded to fp32 and then to the type, lies between the roundings of the true one less and plus
    2^-30."""
    D = 128
    pos, freq = _positions(first), _freq(D)
    x = torch.zeros((pos.numel(), 1, D), dtype=dtype)
    one, zero = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    x[..., one] = 1
    q, _ = lib().qk_norm_rope(x.cuda(), None, pos.cuda(), freq.cuda(), interleaved=interleaved)
    q = q[:, 0].cpu()
    t = pos.double()[:, None] * freq
    for got, want in ((q[:, one], torch.cos(t)), (q[:, zero], torch.sin(t))):
        low, high = ((want + d).float().to(dtype) for d in (-2.0 ** -30, 2.0 ** -30))
        bad = (got < low) | (got > high)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} are roundings of another number"


@pytest.mark.parametrize("first", [0, None], ids=str)
def test_appended_keys_turn_alike(first):
    """The same for keys on their way into a cache."""
    D, page = 64, 128
    pos, freq = _positions(first), _freq(D)
    n = pos.numel()
    x = torch.zeros((n, 1, D), dtype=F16)
    x[..., :D // 2] = 1
    both = torch.zeros((2, n // page, 1, page, D), dtype=F16, device="cuda")
    lib().kv_append(x.cuda(), x.cuda(), both[0], both[1], torch.arange(n).cuda(), positions=pos.cuda(), inv_freq=freq.cuda())
    q, _ = lib().qk_norm_rope(x.cuda(), None, pos.cuda(), freq.cuda())
    assert torch.equal(both[0].reshape(n, 1, D), q)
    assert torch.equal(both[1].reshape(n, 1, D).cpu(), x)
