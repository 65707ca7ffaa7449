"""Prompts that the drafting example's pool does not hold."""
import pytest
import torch

from gpu_support import lib

pytestmark = pytest.mark.gpu


def _prompts(lens, pages, max_len=160):
    lib()
    from hashed_gram_memory_amd import drafting_example as ex
    pool = ex.Pool(len(lens), pages, 8, max_len)
    layer = ex.Layer(ex.random_plan(256), pool, 64, 4, 2, 64)
    g = torch.Generator().manual_seed(3)
    return ex, pool, layer, [torch.randint(0, 64, (n,), generator=g, dtype=torch.int32).cuda() for n in lens]


@pytest.mark.parametrize("lens,pages,max_len,short", [
    ([41, 9], 5, 160, "[1]"),         # the pool holds the first alone
    ([9, 41], 5, 160, "[1]"),         # four pages left over, of the five that it needs
    ([41, 9, 9], 1, 160, "[0, 1, 2]"),
    ([9, 41, 9], 90, 32, "[1]"),      # a table of four pages
])
def test_prompts_without_room_are_refused(lens, pages, max_len, short):
    ex, pool, layer, prompts = _prompts(lens, pages, max_len)
    with pytest.raises(RuntimeError, match="no room for the prompts of the requests " + short.replace("[", r"\[").replace("]", r"\]")):
        ex.prompts_in(layer, prompts)
    assert pool.lengths.tolist() == [0] * len(lens)
    held = [p for row, h in zip(pool.block_table.tolist(), pool.held.tolist()) for p in row[:h]]
    assert sorted(held + pool.free_pages.tolist()[:int(pool.n_free)]) == list(range(pages))
    # with room for what is left of them
    few = [p[:1] for p in prompts]
    last, _ = ex.prompts_in(layer, few)
    assert pool.lengths.tolist() == [0] * len(lens) and last[:, 0].tolist() == [int(p[0]) for p in few]
    assert int(pool.n_free) == pages


def test_prompts_that_just_fit():
    ex, pool, layer, prompts = _prompts([41, 9, 1], 6)
    ex.prompts_in(layer, prompts)
    assert pool.lengths.tolist() == [40, 8, 0] and int(pool.n_free) == 0
