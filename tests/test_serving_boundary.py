"""The serving calls on the host: what they refuse, before anything is launched (no device work)."""
import ctypes
import math

import pytest
import torch

OK, EINVAL, ERANGE, EWORKSPACE, EHIP, EUNSUPPORTED = 0, -1, -2, -3, -4, -5
FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced: validation fails or there is nothing to do
BF16, F16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def sv():
    import hashed_gram_memory_amd.serving as sv
    return sv


@pytest.fixture(scope="module")
def L(sv):
    import hashed_gram_memory_amd as hg
    return hg.lib()


def _set(d, changes):
    for k, v in changes.items():
        setattr(d, k, v)
    return d


def _cache(sv, **changes):
    d = sv.KvCacheDesc(FAKE, FAKE, None, None, 8 * 16 * 128, 8 * 16 * 128, 100, 8, 16, 128, BF16)
    return _set(d, changes)


BAD_CACHES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=FAKE + 8), EINVAL), (dict(v=FAKE + 2), EINVAL),
    (dict(n_pages=0), ERANGE), (dict(n_pages=-1), ERANGE), (dict(n_pages=2 ** 31), ERANGE),
    (dict(n_kv_heads=0), ERANGE), (dict(n_kv_heads=65536), ERANGE),
    (dict(page_size=0), EUNSUPPORTED), (dict(page_size=4), EUNSUPPORTED), (dict(page_size=24), EUNSUPPORTED),
    (dict(page_size=2048), EUNSUPPORTED), (dict(head_dim=96), EUNSUPPORTED), (dict(head_dim=0), EUNSUPPORTED),
    (dict(type=3), EUNSUPPORTED), (dict(k_page_stride=8 * 16 * 128 - 16), EINVAL),
    (dict(v_page_stride=8 * 16 * 128 + 8), EINVAL), (dict(k_page_stride=-8 * 16 * 128), EINVAL),
    (dict(v_page_stride=2 ** 62), EINVAL),
    (dict(type=E4M3), EINVAL), (dict(type=E4M3, k_scale=FAKE), EINVAL),
    (dict(type=E4M3, k_scale=FAKE, v_scale=FAKE + 4), EINVAL),
    (dict(type=F16), EUNSUPPORTED),  # not the type of the call's tensors
]

ROTATION = [(dict(rotary_dim=24), EINVAL), (dict(rotary_dim=144), EINVAL), (dict(positions=None), EINVAL),
            (dict(inv_freq=None), EINVAL), (dict(positions=FAKE + 2), EINVAL), (dict(inv_freq=FAKE + 4), EINVAL),
            (dict(interleaved=2), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
            (dict(eps=math.inf), EINVAL), (dict(reserved0=1), EINVAL), (dict(n_tok=-1), EINVAL),
            (dict(n_tok=2 ** 31), ERANGE), (dict(type=2), EUNSUPPORTED)]


def _norm_rope(sv, **changes):
    d = sv.NormRopeDesc(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, 4096, 128, 1024, 128, 4096, 128, 1024, 128,
                        32, 8, 128, 128, 0, BF16, 1e-6, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", ROTATION + [
    (dict(head_dim=80), EUNSUPPORTED), (dict(n_q_heads=65536), ERANGE), (dict(n_k_heads=2 ** 31), ERANGE),
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(q_out=None), EINVAL), (dict(k_out=FAKE + 8), EINVAL),
    (dict(q=FAKE + 2), EINVAL), (dict(q_weight=FAKE + 8), EINVAL), (dict(k_weight=FAKE + 2), EINVAL),
    (dict(q_token_stride=4100), EINVAL), (dict(k_head_stride=-128), EINVAL), (dict(q_out_head_stride=4), EINVAL),
    (dict(k_out_token_stride=2 ** 40), EINVAL),
], ids=str)
def test_norm_rope_refuses(sv, L, changes, want):
    assert L.engram_qk_norm_rope(ctypes.addressof(_norm_rope(sv, **changes)), None) == want


def test_norm_rope_of_nothing(sv, L):
    assert L.engram_qk_norm_rope(None, None) == EINVAL
    for changes in (dict(n_tok=0), dict(n_tok=0, q=None, k_out=None), dict(n_q_heads=0, n_k_heads=0)):
        assert L.engram_qk_norm_rope(ctypes.addressof(_norm_rope(sv, **changes)), None) == OK


def _append(sv, cache, **changes):
    d = sv.AppendDesc(ctypes.pointer(cache), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, 1024, 128, 1024, 128, 128, 0, BF16,
                      1e-6, 0, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", ROTATION + [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(slots=None), EINVAL), (dict(slots=FAKE + 4), EINVAL),
    (dict(k=FAKE + 8), EINVAL), (dict(v=FAKE + 2), EINVAL), (dict(k_weight=FAKE + 2), EINVAL),
    (dict(k_token_stride=1025), EINVAL), (dict(v_head_stride=-8), EINVAL),
], ids=str)
def test_append_refuses(sv, L, changes, want):
    assert L.engram_kv_append(ctypes.addressof(_append(sv, _cache(sv), **changes)), None) == want


@pytest.mark.parametrize("changes,want", BAD_CACHES, ids=str)
def test_a_bad_cache_is_refused(sv, L, changes, want):
    c = _cache(sv, **changes)
    assert L.engram_kv_append(ctypes.addressof(_append(sv, c)), None) == want
    d = _attention(sv, c)
    need = ctypes.c_size_t(77)
    assert L.engram_paged_attention_workspace(ctypes.addressof(d), ctypes.byref(need)) == want
    assert need.value == 77
    assert L.engram_paged_attention(ctypes.addressof(d), FAKE, 1 << 40, None) == want


def test_append_of_nothing(sv, L):
    assert L.engram_kv_append(None, None) == EINVAL
    d = _append(sv, _cache(sv))
    d.cache = None
    assert L.engram_kv_append(ctypes.addressof(d), None) == EINVAL
    assert L.engram_kv_append(ctypes.addressof(_append(sv, _cache(sv), n_tok=0, k=None, slots=None)), None) == OK


def _attention(sv, cache, **changes):
    d = sv.AttentionDesc(ctypes.pointer(cache), FAKE, FAKE, FAKE, FAKE, FAKE, None, 4, 4, 0, 512, 512, 0, 4096, 128, 4096,
                         128, 32, BF16, 0.1, 0)
    return _set(d, changes)


@pytest.mark.parametrize("changes,want", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(kv_len=None), EINVAL), (dict(block_table=None), EINVAL),
    (dict(q=FAKE + 8), EINVAL), (dict(out=FAKE + 2), EINVAL), (dict(lse=FAKE + 2), EINVAL),
    (dict(kv_len=FAKE + 1), EINVAL), (dict(cu_q=FAKE + 2), EINVAL), (dict(block_table=FAKE + 2), EINVAL),
    (dict(n_seq=-1), EINVAL), (dict(n_seq=0), EINVAL), (dict(n_seq=3), EINVAL), (dict(n_tok=-1), EINVAL),
    (dict(n_seq=(1 << 24) + 1, n_tok=(1 << 24) + 1), ERANGE), (dict(n_tok=2 ** 27), ERANGE),
    (dict(n_tok=1 << 23, n_seq=1 << 23), ERANGE),
    (dict(table_width=-1), EINVAL), (dict(table_stride=511), EINVAL), (dict(table_stride=-512), EINVAL),
    (dict(table_width=2 ** 31, table_stride=2 ** 31), ERANGE), (dict(max_q_len=-1), EINVAL),
    (dict(window=-1), EINVAL), (dict(window=2 ** 31), ERANGE),
    (dict(n_q_heads=0), EINVAL), (dict(n_q_heads=12), EINVAL), (dict(n_q_heads=65536), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(reserved0=1), EINVAL),
    (dict(type=E4M3), EUNSUPPORTED), (dict(type=5), EUNSUPPORTED),
    (dict(q_token_stride=4097), EINVAL), (dict(q_head_stride=-128), EINVAL), (dict(out_token_stride=4), EINVAL),
    (dict(out_head_stride=2 ** 41), EINVAL),
], ids=str)
def test_attention_refuses(sv, L, changes, want):
    d = _attention(sv, _cache(sv), **changes)
    assert L.engram_paged_attention(ctypes.addressof(d), FAKE, 1 << 40, None) == want


def test_attention_workspace(sv, L):
    need = ctypes.c_size_t(77)
    d = _attention(sv, _cache(sv))
    at = ctypes.addressof(d)
    assert L.engram_paged_attention_workspace(None, ctypes.byref(need)) == EINVAL
    assert L.engram_paged_attention_workspace(at, None) == EINVAL
    assert L.engram_paged_attention(None, None, 0, None) == EINVAL
    assert L.engram_paged_attention_workspace(at, ctypes.byref(need)) == OK
    assert need.value > 0  # 4 requests of up to 8,192 keys: divided
    for ws, n in ((None, need.value), (FAKE, need.value - 1), (FAKE + 128, need.value)):
        assert L.engram_paged_attention(at, ws, n, None) == EWORKSPACE
    # a few keys are not divided, and no token needs nothing
    for changes in (dict(table_width=4), dict(n_tok=0), dict(n_tok=0, n_seq=0, q=None, kv_len=None)):
        d = _attention(sv, _cache(sv), **changes)
        assert L.engram_paged_attention_workspace(ctypes.addressof(d), ctypes.byref(need)) == OK
        assert need.value == 0
    d = _attention(sv, _cache(sv), n_tok=0)
    assert L.engram_paged_attention(ctypes.addressof(d), None, 0, None) == OK


def test_binding_refuses_host_tensors():
    import hashed_gram_memory_amd as hg
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    cache = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hg.qk_norm_rope(q, None)
    with pytest.raises(ValueError):
        hg.kv_append(q[:, :2], q[:, :2], cache, cache, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        hg.paged_attention(q, cache, cache, torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        hg.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        hg.qk_norm_rope(q.float(), None)
