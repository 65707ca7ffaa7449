"""The calls of a drafting step on the host: what they refuse, before anything is launched (no device work)."""
import ctypes
import math
import random

import pytest
import torch

from test_serving_boundary import (BAD_CACHES, EINVAL, ERANGE, EUNSUPPORTED, EWORKSPACE, FAKE, OK, ROTATION, _attention, _cache,
                                   _set)

BF16, F16, E4M3, E4M3_PAGE, I8_PAGE, F32 = 0, 1, 2, 4, 5, 6


@pytest.fixture(scope="module")
def sv():
    from hashed_gram_memory_amd import serving
    return serving


@pytest.fixture(scope="module")
def L(sv):
    import hashed_gram_memory_amd as hg
    return hg.lib()


def _pages(sv, **changes):
    return _set(_cache(sv, type=I8_PAGE, k_scale=FAKE, v_scale=FAKE), changes)


def _append(sv, cache, **changes):
    d = sv.AppendPagesDesc(ctypes.pointer(cache), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 0, 512, 512, 1024, 128,
                           1024, 128, 128, 0, BF16, 1e-6, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", [x for x in ROTATION if x[0] != dict(n_tok=2 ** 31)] + [
    (dict(n_tok=2 ** 31), ERANGE), (dict(type=I8_PAGE), EUNSUPPORTED),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(block_table=None), EINVAL), (dict(kv_len=None), EINVAL),
    (dict(k=FAKE + 8), EINVAL), (dict(v=FAKE + 2), EINVAL), (dict(k_weight=FAKE + 2), EINVAL), (dict(block_table=FAKE + 2), EINVAL),
    (dict(kv_len=FAKE + 1), EINVAL), (dict(cu_q=FAKE + 2), EINVAL), (dict(n_seq=-1), EINVAL), (dict(n_seq=0), EINVAL),
    (dict(cu_q=None, n_seq=3), EINVAL), (dict(n_seq=(1 << 24) + 1), ERANGE), (dict(max_q_len=-1), EINVAL),
    (dict(table_width=-1), EINVAL), (dict(table_stride=511), EINVAL), (dict(table_stride=-1), EINVAL),
    (dict(table_width=2 ** 31, table_stride=2 ** 31), ERANGE), (dict(k_token_stride=1025), EINVAL), (dict(v_head_stride=-8), EINVAL),
    (dict(n_seq=1 << 23, n_tok=1 << 23), ERANGE), (dict(n_seq=1 << 21, n_tok=1 << 21, max_q_len=1), ERANGE),
    (dict(n_tok=2 ** 31 - 1), ERANGE),
], ids=str)
def test_append_pages_refuses(sv, L, changes, want):
    assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, _pages(sv), **changes)), None) == want


@pytest.mark.parametrize("kind", [E4M3_PAGE, I8_PAGE])
@pytest.mark.parametrize("changes,want", [x for x in BAD_CACHES if "type" not in x[0]] + [
    (dict(k_scale=None), EINVAL), (dict(v_scale=None), EINVAL), (dict(v_scale=FAKE + 4), EINVAL)], ids=str)
def test_a_bad_cache_is_refused(sv, L, kind, changes, want):
    c = _set(_pages(sv, type=kind), changes)
    assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, c)), None) == want
    d = _attention(sv, c)
    assert L.engram_paged_attention(ctypes.addressof(d), FAKE, 1 << 40, None) == want


def test_appends_and_the_caches_that_they_take(sv, L):
    """A scale for each row, or none, goes with one append, a scale for each page with the other."""
    for kind in (BF16, F16, E4M3, 3, F32, 7):
        c = _cache(sv, type=kind, k_scale=FAKE, v_scale=FAKE)
        assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, c)), None) == EUNSUPPORTED
    for kind in (E4M3_PAGE, I8_PAGE):
        c = _cache(sv, type=kind, k_scale=FAKE, v_scale=FAKE)
        d = sv.AppendDesc(ctypes.pointer(c), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, 1024, 128, 1024, 128, 128, 0, BF16, 1e-6, 0, 0)
        assert L.engram_kv_append(ctypes.addressof(d), None) == EUNSUPPORTED
        need = ctypes.c_size_t(0)
        for q in (BF16, F16):
            assert L.engram_paged_attention_workspace(ctypes.addressof(_attention(sv, c, type=q)), ctypes.byref(need)) == OK


def test_append_pages_of_nothing(sv, L):
    assert L.engram_kv_append_pages(None, None) == EINVAL
    d = _append(sv, _pages(sv))
    d.cache = None
    assert L.engram_kv_append_pages(ctypes.addressof(d), None) == EINVAL
    for changes in (dict(n_tok=0), dict(n_tok=0, n_seq=0, k=None, block_table=None), dict(table_width=0, block_table=None)):
        assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, _pages(sv), **changes)), None) == OK


def _tables(sv, **changes):
    d = sv.PageTablesDesc(*[FAKE] * 11, 4, 8, 32, 32, 100, 16, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", [
    *[(dict([(f, None)]), EINVAL) for f in ("lengths", "block_table", "held", "free_pages", "n_free", "slots", "positions", "cu_q",
                                            "kv_len", "n_short")],
    *[(dict([(f, FAKE + 2)]), EINVAL) for f in ("lengths", "new_tokens", "block_table", "held", "free_pages", "n_free", "positions",
                                                "cu_q", "kv_len", "n_short")],
    (dict(slots=FAKE + 4), EINVAL), (dict(n_seq=-1), EINVAL), (dict(n_tok=-1), EINVAL), (dict(table_width=-1), EINVAL),
    (dict(n_pages=-1), EINVAL), (dict(reserved0=1), EINVAL), (dict(table_stride=31), EINVAL), (dict(table_stride=-32), EINVAL),
    (dict(page_size=0), EUNSUPPORTED), (dict(page_size=4), EUNSUPPORTED), (dict(page_size=24), EUNSUPPORTED),
    (dict(page_size=2048), EUNSUPPORTED), (dict(n_seq=(1 << 20) + 1), ERANGE), (dict(n_tok=1 << 30), ERANGE),
    (dict(table_width=2 ** 31, table_stride=2 ** 31), ERANGE), (dict(n_pages=(1 << 30) + 1), ERANGE),
    (dict(new_tokens=None, n_seq=3), EINVAL),
], ids=str)
def test_page_tables_refuses(sv, L, changes, want):
    d = _tables(sv, **changes)
    need = ctypes.c_size_t(77)
    assert L.engram_page_tables_workspace(ctypes.addressof(d), ctypes.byref(need)) == want and need.value == 77
    assert L.engram_page_tables(ctypes.addressof(d), FAKE, 1 << 40, None) == want


def test_page_tables_workspace(sv, L):
    need = ctypes.c_size_t(77)
    assert L.engram_page_tables_workspace(None, ctypes.byref(need)) == EINVAL
    assert L.engram_page_tables_workspace(ctypes.addressof(_tables(sv)), None) == EINVAL
    assert L.engram_page_tables(None, None, 0, None) == EINVAL
    assert L.engram_page_tables_workspace(ctypes.addressof(_tables(sv)), ctypes.byref(need)) == OK and need.value == 0
    rng = random.Random(2)
    for _ in range(200):
        n, t = rng.choice([1025, 4096, 1 << 20]), rng.choice([0, 9000, (1 << 30) - 1])
        d = _tables(sv, n_seq=n, n_tok=t)
        assert L.engram_page_tables_workspace(ctypes.addressof(d), ctypes.byref(need)) == OK
        assert need.value >= 12 * n and need.value % 256 == 0
        for ws, size in ((None, need.value), (FAKE, need.value - 1), (FAKE + 128, need.value)):
            assert L.engram_page_tables(ctypes.addressof(d), ws, size, None) == EWORKSPACE


def _verify(sv, **changes):
    d = sv.VerifyDraftDesc(*[FAKE] * 8, 4, 8, 50000, 50000, 50000, F32, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", [
    *[(dict([(f, None)]), EINVAL) for f in ("target", "draft", "uniform", "last_uniform", "tokens", "n_accepted")],
    *[(dict([(f, FAKE + 2)]), EINVAL) for f in ("target", "draft_probs", "draft", "uniform", "last_uniform", "cu_draft", "tokens",
                                                "n_accepted")],
    (dict(type=BF16, target=FAKE + 1), EINVAL), (dict(type=E4M3), EUNSUPPORTED), (dict(type=7), EUNSUPPORTED),
    (dict(n_seq=-1), EINVAL), (dict(n_draft=-1), EINVAL), (dict(vocab=-1), EINVAL), (dict(vocab=0), EINVAL), (dict(reserved0=1), EINVAL),
    (dict(n_seq=0), EINVAL), (dict(cu_draft=None, n_seq=3), EINVAL), (dict(target_stride=-1), EINVAL),
    (dict(draft_stride=2 ** 41), EINVAL), (dict(n_seq=(1 << 20) + 1), ERANGE), (dict(n_draft=(1 << 30) + 1), ERANGE),
    (dict(vocab=(1 << 30) + 1), ERANGE), (dict(n_seq=1 << 20), ERANGE),
], ids=str)
def test_verify_draft_refuses(sv, L, changes, want):
    d = _verify(sv, **changes)
    need = ctypes.c_size_t(77)
    assert L.engram_verify_draft_workspace(ctypes.addressof(d), ctypes.byref(need)) == want and need.value == 77
    assert L.engram_verify_draft(ctypes.addressof(d), FAKE, 1 << 40, None) == want


def test_verify_draft_workspace(sv, L):
    need = ctypes.c_size_t(77)
    assert L.engram_verify_draft_workspace(None, ctypes.byref(need)) == EINVAL
    assert L.engram_verify_draft(None, None, 0, None) == EINVAL
    d = _verify(sv)
    assert L.engram_verify_draft_workspace(ctypes.addressof(d), None) == EINVAL
    assert L.engram_verify_draft_workspace(ctypes.addressof(d), ctypes.byref(need)) == OK and need.value > 0
    for ws, size in ((None, need.value), (FAKE, need.value - 1), (FAKE + 128, need.value)):
        assert L.engram_verify_draft(ctypes.addressof(d), ws, size, None) == EWORKSPACE
    for changes in (dict(vocab=1000), dict(n_seq=0, n_draft=0, target=None)):
        assert L.engram_verify_draft_workspace(ctypes.addressof(_verify(sv, **changes)), ctypes.byref(need)) == OK and need.value == 0
    assert L.engram_verify_draft(ctypes.addressof(_verify(sv, n_seq=0, n_draft=0)), None, 0, None) == OK


def test_reserved_field_of_append_pages(sv, L):
    assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, _pages(sv), reserved0=1)), None) == EINVAL
    assert L.engram_kv_append_pages(ctypes.addressof(_append(sv, _pages(sv), eps=math.inf)), None) == EINVAL


def test_binding_refuses_host_tensors():
    import hashed_gram_memory_amd as hg
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    cache, scale = torch.zeros((2, 2, 16, 64), dtype=torch.int8), torch.zeros((2, 2))
    table, one = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        hg.kv_append_pages(k, k, cache, cache, scale, scale, table, one)
    with pytest.raises(ValueError, match="device tensor"):
        hg.page_tables(one, one, table, one, one, one, 16, 1)
    with pytest.raises(ValueError, match="device tensor"):
        hg.verify_draft(torch.ones((2, 5)), one, torch.zeros(1), torch.zeros(1))
    with pytest.raises(TypeError):
        hg.verify_draft(None, one, one, one)
