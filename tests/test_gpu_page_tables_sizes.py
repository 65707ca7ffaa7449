"""Sizes of page_tables past its limits: refused before anything is allocated for them."""
import pytest
import torch

from gpu_support import lib

pytestmark = pytest.mark.gpu


def _args(n_seq=2, width=3, n_pages=9):
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return z(n_seq), z(n_seq) + 1, z(n_seq, width), z(n_seq), torch.arange(n_pages, dtype=torch.int32, device="cuda"), z(1) + n_pages


@pytest.mark.parametrize("n_tok", [2 ** 30, 2 ** 31, 2 ** 36, 2 ** 40, 2 ** 60, 2 ** 61, 2 ** 62, 2 ** 63 - 1])
def test_batches_past_the_limit(n_tok):
    hg = lib()
    args = _args()
    before = [x.clone() for x in args]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for call in (lambda: hg.page_tables(*args, 16, n_tok), lambda: hg.page_tables_workspace(*args, 16, n_tok)):
        with pytest.raises(hg.EngramError) as e:
            call()
        assert e.value.status == -2  # ENGRAM_ERANGE
    assert torch.cuda.max_memory_allocated() == held
    assert all(torch.equal(x, y) for x, y in zip(args, before))


def test_numbers_that_are_no_int64():
    hg = lib()
    for n_tok in (2 ** 63, -2 ** 63 - 1):
        with pytest.raises(OverflowError):
            hg.page_tables(*_args(), 16, n_tok)
    with pytest.raises(ValueError):
        hg.page_tables(*_args(), 16, -1)
