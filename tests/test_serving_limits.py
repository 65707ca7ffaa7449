"""Descriptions of paged attention at their limits (host side; no GPU): every one ends with a status."""
import ctypes
import random

import pytest

from test_serving_boundary import EINVAL, ERANGE, EUNSUPPORTED, OK, _attention, _cache


@pytest.fixture(scope="module")
def sv():
    from hashed_gram_memory_amd import serving
    return serving


@pytest.fixture(scope="module")
def L(sv):
    import hashed_gram_memory_amd as hg
    return hg.lib()


@pytest.mark.parametrize("tokens", [4, 4096])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_a_table_without_pages(sv, L, tokens, head_dim):
    need = ctypes.c_size_t(77)
    stride = 16 * head_dim * 8
    cache = _cache(sv, head_dim=head_dim, k_page_stride=stride, v_page_stride=stride)
    d = _attention(sv, cache, table_width=0, table_stride=0, block_table=None, n_tok=tokens)
    assert L.engram_paged_attention_workspace(ctypes.addressof(d), ctypes.byref(need)) == OK
    assert need.value == 0


def test_workspaces_over_the_range(sv, L):
    """The same for random sizes, the largest of each among them."""
    rng = random.Random(1)
    pick = lambda *x: rng.choice(x)  # noqa: E731
    seen = set()
    for _ in range(4000):
        dim = pick(64, 128, 256)
        page = pick(8, 16, 1024)
        heads = pick(1, 2, 8, 65535)
        stride = page * dim * heads
        cache = _cache(sv, n_kv_heads=heads, page_size=page, head_dim=dim, k_page_stride=stride, v_page_stride=stride)
        n_seq = pick(1, 3, 64, 1 << 24)
        width = pick(0, 1, 512, 2 ** 31 - 1)
        d = _attention(sv, cache, n_seq=n_seq, n_tok=n_seq * pick(1, 2, 17, 300, 1 << 20), table_width=width,
                       table_stride=width, n_q_heads=min(65535, heads * pick(1, 4, 40)),
                       cu_q=pick(None, 1 << 20), max_q_len=pick(0, 1, 9, 2 ** 31), window=pick(0, 1, 1024, 2 ** 31 - 1))
        need = ctypes.c_size_t(0)
        st = L.engram_paged_attention_workspace(ctypes.addressof(d), ctypes.byref(need))
        assert st in (OK, EINVAL, ERANGE, EUNSUPPORTED)
        assert need.value % 256 == 0
        seen.add(st)
    assert OK in seen and ERANGE in seen
