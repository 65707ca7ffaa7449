"""Serving operators next to the lookup: head norm + rotation, paged cache append, paged attention.

Argument marshalling only, as in the package's own module; the C ABI is in
include/engram.h.  A cache is a pair of device tensors [n_pages, n_kv_heads,
page_size, head_dim] that the caller owns: bfloat16 or float16, or FP8 E4M3
codes (uint8 or float8_e4m3fn) with float32 scales [n_pages, n_kv_heads,
page_size] for K and V.

    q, _ = qk_norm_rope(q, None, positions, inv_freq, q_weight=wq)       # engram_qk_norm_rope
    kv_append(k, v, k_cache, v_cache, slots, positions=positions, inv_freq=inv_freq, k_weight=wk)  # engram_kv_append
    out = paged_attention(q, k_cache, v_cache, block_table, kv_len)       # engram_paged_attention

attention_example.py runs them together, next to the lookup.

The operators serve: they have no backward, and refuse tensors that require
a gradient while gradients are recorded, and those with a forward gradient.  They run on the current stream of
their tensors' device, or on ``stream``, a stream or handle of that device.  The calls are marshalled by the
extension _serving.so (csrc/serving_binding.cpp); the ctypes structures below are
the C ABI's descriptions, for callers that hold plain pointers.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

import hashed_gram_memory_amd as _hg

_VP, _I64, _U32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float

BF16, F16, E4M3 = 0, 1, 2


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("k_page_stride", _I64),
                ("v_page_stride", _I64), ("n_pages", _I64), ("n_kv_heads", _U32), ("page_size", _U32),
                ("head_dim", _U32), ("type", _U32)]


class NormRopeDesc(ctypes.Structure):
    _fields_ = [("q", _VP), ("k", _VP), ("q_out", _VP), ("k_out", _VP), ("q_weight", _VP), ("k_weight", _VP),
                ("positions", _VP), ("inv_freq", _VP), ("n_tok", _I64),
                ("q_token_stride", _I64), ("q_head_stride", _I64), ("k_token_stride", _I64), ("k_head_stride", _I64),
                ("q_out_token_stride", _I64), ("q_out_head_stride", _I64), ("k_out_token_stride", _I64),
                ("k_out_head_stride", _I64), ("n_q_heads", _U32), ("n_k_heads", _U32), ("head_dim", _U32),
                ("rotary_dim", _U32), ("interleaved", _U32), ("type", _U32), ("eps", _F32), ("reserved0", _U32)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(KvCacheDesc)), ("k", _VP), ("v", _VP), ("k_weight", _VP), ("positions", _VP),
                ("inv_freq", _VP), ("slots", _VP), ("n_tok", _I64), ("k_token_stride", _I64), ("k_head_stride", _I64),
                ("v_token_stride", _I64), ("v_head_stride", _I64), ("rotary_dim", _U32), ("interleaved", _U32),
                ("type", _U32), ("eps", _F32), ("reserved0", _U32), ("reserved1", _U32)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(KvCacheDesc)), ("q", _VP), ("out", _VP), ("lse", _VP), ("block_table", _VP),
                ("kv_len", _VP), ("cu_q", _VP), ("n_seq", _I64), ("n_tok", _I64), ("max_q_len", _I64),
                ("table_width", _I64), ("table_stride", _I64), ("window", _I64), ("q_token_stride", _I64),
                ("q_head_stride", _I64), ("out_token_stride", _I64), ("out_head_stride", _I64), ("n_q_heads", _U32),
                ("type", _U32), ("scale", _F32), ("reserved0", _U32)]


_lib = _hg.lib()
for _name, _args in {"engram_qk_norm_rope": [_VP, _VP], "engram_kv_append": [_VP, _VP],
                     "engram_paged_attention_workspace": [_VP, ctypes.POINTER(ctypes.c_size_t)],
                     "engram_paged_attention": [_VP, _VP, ctypes.c_size_t, _VP]}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = ctypes.c_int

if not os.path.exists(os.path.join(os.path.dirname(__file__), "_serving.so")):
    raise ImportError("_serving.so is not built; run `python hashed_gram_memory_amd/build.py`")
from . import _serving  # noqa: E402

_serving.setup(_hg.EngramError, torch._C._cuda_getCurrentRawStream, torch.OutOfMemoryError)


def _on(stream, lead):
    """``stream`` (a torch.cuda.Stream or a handle; 0: the default one) as the current one of the device of ``lead``, the
    call's first tensor: outputs come from its pool, so that they are not reused while work is queued."""
    device = getattr(lead, "device", None)
    if device is None or device.type != "cuda":
        return contextlib.nullcontext()  # the call refuses it
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        # a pointer of 0 would be taken for none given, and get a new stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is one of {stream.device}, not of {device}")
    return torch.cuda.stream(stream)


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """RMS norm of every head of ``q`` [n_tok, n_q_heads, head_dim] and ``k`` [n_tok, n_k_heads, head_dim] (where its
    weight [head_dim] is given) and their rotation by ``positions`` int32 [n_tok] (where ``inv_freq`` float64
    [rotary_dim / 2] is given), in one pass: (q_out, k_out) (engram_qk_norm_rope).  Either side may be None; an output
    may be its input."""
    args = (q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    if stream is None:
        return _serving.qk_norm_rope(*args)
    with _on(stream, k if q is None else q):
        return _serving.qk_norm_rope(*args)


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
              positions: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None,
              k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
              k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None, stream=None) -> None:
    """Write new keys (normed and rotated as in qk_norm_rope) and values [n_tok, n_kv_heads, head_dim] to the cache's
    ``slots`` int64 [n_tok] (page * page_size + place; a negative slot is skipped) (engram_kv_append)."""
    args = (k, v, k_cache, v_cache, slots, positions, inv_freq, k_weight, eps, interleaved, k_scale, v_scale)
    if stream is None:
        return _serving.kv_append(*args)
    with _on(stream, k):
        return _serving.kv_append(*args)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    kv_len: torch.Tensor, cu_q: torch.Tensor | None = None, max_q_len: int | None = None,
                    scale: float | None = None, window: int = 0, k_scale: torch.Tensor | None = None,
                    v_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, return_lse: bool = False,
                    workspace: torch.Tensor | None = None, stream=None):
    """Causal attention of new tokens ``q`` [n_tok, n_q_heads, head_dim] over a paged cache that holds them: ``out`` of
    q's shape, with ``return_lse`` (out, lse float32 [n_tok, n_q_heads]) (engram_paged_attention).

    Request b has tokens cu_q[b] .. cu_q[b+1]-1 (int32 [n_seq + 1]; None: equally many each; tokens from cu_q[n_seq] on
    are no request's, and their rows of the outputs are not written) and kv_len[b] cached keys
    (int32 [n_seq]) on the pages block_table[b] (int32 [n_seq, width]).  ``max_q_len`` bounds the tokens of a request
    where it is known: a batch of single tokens takes fewer launches with it, and a request that is longer may be left
    out.  Softmax weights are held in about 16 bits where a request has at most 32 rows (tokens * query heads of a key)
    and are rounded once to q's type where it has more, which adds to the output about what its own rounding does.  ``scale`` defaults to head_dim ** -0.5; ``window`` > 0 lets a token see that many keys.
    ``workspace``: uint8 of paged_attention_workspace bytes, 256-byte aligned; allocated if not given."""
    args = (q, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len, scale, window, k_scale, v_scale, out, return_lse,
            workspace, False)
    if stream is None:
        return _serving.paged_attention(*args)
    with _on(stream, q):
        return _serving.paged_attention(*args)


def paged_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                              kv_len: torch.Tensor, cu_q: torch.Tensor | None = None, max_q_len: int | None = None,
                              window: int = 0, k_scale: torch.Tensor | None = None,
                              v_scale: torch.Tensor | None = None) -> int:
    """Bytes of the workspace that paged_attention needs with these arguments; it goes by their shapes, ``max_q_len`` and
    ``window`` alone (engram_paged_attention_workspace)."""
    return _serving.paged_attention(q, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len, None, window, k_scale, v_scale,
                                    None, False, None, True)
