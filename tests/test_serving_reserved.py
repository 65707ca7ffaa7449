"""Every reserved field of the serving calls' descriptions must be 0 (host side; no GPU)."""
import ctypes

import pytest

from test_serving_boundary import EINVAL, _append, _attention, _cache, _norm_rope


@pytest.mark.parametrize("call,make", [
    ("engram_qk_norm_rope", lambda sv, **c: _norm_rope(sv, **c)),
    ("engram_kv_append", lambda sv, **c: _append(sv, _cache(sv), **c)),
    ("engram_paged_attention", lambda sv, **c: _attention(sv, _cache(sv), **c)),
], ids=["qk_norm_rope", "kv_append", "paged_attention"])
def test_reserved_fields(call, make):
    import hashed_gram_memory_amd as hg
    from hashed_gram_memory_amd import serving as sv

    fields = [f for f, _ in make(sv)._fields_ if f.startswith("reserved")]
    assert fields
    for f in fields:
        d = make(sv, **{f: 1})
        more = (None, 0, None) if call == "engram_paged_attention" else (None,)
        assert getattr(hg.lib(), call)(ctypes.addressof(d), *more) == EINVAL, f
