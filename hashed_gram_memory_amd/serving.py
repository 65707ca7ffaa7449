"""Serving operators next to the lookup: head norm + rotation, paged cache append, paged attention.

Argument marshalling only, as in the package's own module; the C ABI is in
include/engram.h.  A cache is a pair of device tensors [n_pages, n_kv_heads,
page_size, head_dim] that the caller owns: bfloat16 or float16, or FP8 E4M3
codes (uint8 or float8_e4m3fn) with float32 scales [n_pages, n_kv_heads,
page_size] for K and V.

    q, _ = qk_norm_rope(q, None, positions, inv_freq, q_weight=wq)       # engram_qk_norm_rope
    kv_append(k, v, k_cache, v_cache, slots, positions=positions, inv_freq=inv_freq, k_weight=wk)  # engram_kv_append
    out = paged_attention(q, k_cache, v_cache, block_table, kv_len)       # engram_paged_attention

The operators serve: they have no backward, and refuse tensors that require
a gradient while gradients are recorded.
"""
from __future__ import annotations

import ctypes

import torch

import hashed_gram_memory_amd as _hg

_VP, _I64, _U32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float

BF16, F16, E4M3 = 0, 1, 2
_TYPES = {torch.bfloat16: BF16, torch.float16: F16}
_CACHE_TYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}


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


def _device(t, device, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and the operator has no backward")


def _rows(t, device, dtype, name: str, dim: int = 0):
    """Pointer and token and head strides of a [n_tok, heads, dim] tensor; a stride of an axis of one is 0."""
    _device(t, device, name)
    if t.dim() != 3 or t.dtype != dtype or (dim and t.shape[2] != dim):
        raise ValueError(f"{name} must be a {dtype} tensor [n_tok, heads, {dim or 'head_dim'}], got {t.dtype} "
                         f"{list(t.shape)}")
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous along head_dim")
    return t.data_ptr(), st if n > 1 else 0, sh if h > 1 else 0


def _out_rows(t, device, dtype, shape, name: str):
    """As _rows, for an output: of that shape, with no two elements in one place."""
    if isinstance(t, torch.Tensor) and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    ptr, st, sh = _rows(t, device, dtype, name)
    n, h, d = shape
    inner, outer = sorted(((sh, h), (st, n)))
    if (inner[1] > 1 and inner[0] < d) or (outer[1] > 1 and outer[0] < max(inner[0] * inner[1], d)):
        raise ValueError(f"{name} has overlapping rows (strides {t.stride()})")
    return ptr, st, sh


def _vector(t, device, dtype, n: int, name: str) -> int | None:
    if t is None:
        return None
    _device(t, device, name)
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n}], got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for work on ``stream``: taken from that stream's pool, so that it is not reused while work is queued."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rotation(positions, inv_freq, n_tok: int, device):
    """(positions, inv_freq, rotary_dim); without inv_freq nothing is rotated."""
    if inv_freq is None:
        return None, None, 0
    _device(inv_freq, device, "inv_freq")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 [rotary_dim / 2]")
    if positions is None:
        raise ValueError("inv_freq needs positions")
    return _vector(positions, device, torch.int32, n_tok, "positions"), inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def _cache_axis(t, device, name: str):
    _device(t, device, name)
    if t.dim() != 4 or t.dtype not in _CACHE_TYPES:
        raise ValueError(f"{name} must be a bfloat16, float16, uint8 or float8_e4m3fn tensor "
                         f"[n_pages, n_kv_heads, page_size, head_dim], got {t.dtype} {list(t.shape)}")
    n, h, p, d = t.shape
    sn, sh, sp, sd = t.stride()
    if (sd != 1 and d > 1) or (sp != d and p > 1) or (sh != p * d and h > 1):
        raise ValueError(f"{name} must have contiguous pages")
    return t.data_ptr(), sn if n > 1 else h * p * d


def _cache(k_cache, v_cache, k_scale, v_scale, device) -> KvCacheDesc:
    k, ks = _cache_axis(k_cache, device, "k_cache")
    v, vs = _cache_axis(v_cache, device, "v_cache")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same shape and type")
    kind = _CACHE_TYPES[k_cache.dtype]
    scales = [None, None]
    if kind == E4M3:
        for i, (t, name) in enumerate(((k_scale, "k_scale"), (v_scale, "v_scale"))):
            if t is None:
                raise ValueError(f"an e4m3 cache needs {name}")
            _device(t, device, name)
            if t.dtype != torch.float32 or t.shape != k_cache.shape[:3] or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 {list(k_cache.shape[:3])}")
            scales[i] = t.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to an e4m3 cache")
    n, h, p, d = k_cache.shape
    return KvCacheDesc(k, v, scales[0], scales[1], ks, vs, n, h, p, d, kind)


def _type(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _TYPES[t.dtype]


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """RMS norm of every head of ``q`` [n_tok, n_q_heads, head_dim] and ``k`` [n_tok, n_k_heads, head_dim] (where its
    weight [head_dim] is given) and their rotation by ``positions`` int32 [n_tok] (where ``inv_freq`` float64
    [rotary_dim / 2] is given), in one pass: (q_out, k_out) (engram_qk_norm_rope).  Either side may be None; an output
    may be its input."""
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is needed")
    kind = _type(lead, "q" if q is not None else "k")
    device, dtype = lead.device, lead.dtype
    if lead.dim() != 3:
        raise ValueError("q and k must be [n_tok, heads, head_dim]")
    n_tok, _, dim = lead.shape
    side = []
    for x, w, out, name in ((q, q_weight, q_out, "q"), (k, k_weight, k_out, "k")):
        if x is None:
            if w is not None or out is not None:
                raise ValueError(f"{name}_weight and {name}_out need {name}")
            side.append((None, 0, 0, None, 0, 0, None, 0, None))
            continue
        src = _rows(x, device, dtype, name, dim)
        if x.shape[0] != n_tok:
            raise ValueError("q and k must have the same tokens")
        if out is None:
            out = _empty(x.shape, dtype, device, stream)
            dst = out.data_ptr(), x.shape[1] * dim, dim
        else:
            dst = _out_rows(out, device, dtype, x.shape, name + "_out")
        side.append((*src, *dst, _vector(w, device, dtype, dim, name + "_weight"), x.shape[1], out))
    pos, freq, rotary = _rotation(positions, inv_freq, n_tok, device)
    a, b = side
    d = NormRopeDesc(a[0], b[0], a[3], b[3], a[6], b[6], pos, freq, n_tok, a[1], a[2], b[1], b[2], a[4], a[5], b[4],
                     b[5], a[7], b[7], dim, rotary, bool(interleaved), kind, eps, 0)
    _hg._check(_lib.engram_qk_norm_rope(ctypes.addressof(d), _hg._stream(stream)), "engram_qk_norm_rope")
    return a[8], b[8]


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
              positions: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None,
              k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
              k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None, stream=None) -> None:
    """Write new keys (normed and rotated as in qk_norm_rope) and values [n_tok, n_kv_heads, head_dim] to the cache's
    ``slots`` int64 [n_tok] (page * page_size + place; a negative slot is skipped) (engram_kv_append)."""
    kind = _type(k, "k")
    device, dtype = k.device, k.dtype
    c = _cache(k_cache, v_cache, k_scale, v_scale, device)
    kr = _rows(k, device, dtype, "k", c.head_dim)
    vr = _rows(v, device, dtype, "v", c.head_dim)
    if k.shape != v.shape or k.shape[1] != c.n_kv_heads:
        raise ValueError(f"k and v must be [n_tok, {c.n_kv_heads}, {c.head_dim}]")
    n_tok = k.shape[0]
    at = _vector(slots, device, torch.int64, n_tok, "slots")
    if at is None:
        raise TypeError("slots must be a torch.Tensor")
    w = _vector(k_weight, device, dtype, c.head_dim, "k_weight")
    pos, freq, rotary = _rotation(positions, inv_freq, n_tok, device)
    d = AppendDesc(ctypes.pointer(c), kr[0], vr[0], w, pos, freq, at, n_tok, kr[1], kr[2], vr[1], vr[2], rotary,
                   bool(interleaved), kind, eps, 0, 0)
    _hg._check(_lib.engram_kv_append(ctypes.addressof(d), _hg._stream(stream)), "engram_kv_append")


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    kv_len: torch.Tensor, cu_q: torch.Tensor | None = None, max_q_len: int | None = None,
                    scale: float | None = None, window: int = 0, k_scale: torch.Tensor | None = None,
                    v_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, return_lse: bool = False,
                    workspace: torch.Tensor | None = None, stream=None):
    """Causal attention of new tokens ``q`` [n_tok, n_q_heads, head_dim] over a paged cache that holds them: ``out`` of
    q's shape, with ``return_lse`` (out, lse float32 [n_tok, n_q_heads]) (engram_paged_attention).

    Request b has tokens cu_q[b] .. cu_q[b+1]-1 (int32 [n_seq + 1]; None: equally many each) and kv_len[b] cached keys
    (int32 [n_seq]) on the pages block_table[b] (int32 [n_seq, width]).  ``max_q_len`` bounds the tokens of a request
    where it is known.  ``scale`` defaults to head_dim ** -0.5; ``window`` > 0 lets a token see that many keys.
    ``workspace``: uint8 of the bytes that engram_paged_attention_workspace asks for, 256-byte aligned; allocated
    if not given."""
    kind = _type(q, "q")
    device, dtype = q.device, q.dtype
    c = _cache(k_cache, v_cache, k_scale, v_scale, device)
    qr = _rows(q, device, dtype, "q", c.head_dim)
    n_tok, heads, dim = q.shape
    _device(block_table, device, "block_table")
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [n_seq, width]")
    n_seq, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must be contiguous along its width")
    lens = _vector(kv_len, device, torch.int32, n_seq, "kv_len")
    if lens is None:
        raise TypeError("kv_len must be a torch.Tensor")
    cu = _vector(cu_q, device, torch.int32, n_seq + 1, "cu_q")
    if out is None:
        out = _empty(q.shape, dtype, device, stream)
        dst = out.data_ptr(), heads * dim, dim
    else:
        dst = _out_rows(out, device, dtype, q.shape, "out")
    lse = _empty((n_tok, heads), torch.float32, device, stream) if return_lse else None
    d = AttentionDesc(ctypes.pointer(c), qr[0], dst[0], None if lse is None else lse.data_ptr(), block_table.data_ptr(),
                      lens, cu, n_seq, n_tok, 0 if max_q_len is None else max_q_len, width,
                      block_table.stride(0) if n_seq > 1 else width, window, qr[1], qr[2], dst[1], dst[2], heads, kind,
                      dim ** -0.5 if scale is None else scale, 0)
    need = ctypes.c_size_t()
    at = ctypes.addressof(d)
    _hg._check(_lib.engram_paged_attention_workspace(at, ctypes.byref(need)), "engram_paged_attention_workspace")
    ws = ws_bytes = None
    if workspace is not None:
        _device(workspace, device, "workspace")
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    elif need.value:
        workspace = _empty((need.value,), torch.uint8, device, stream)
        ws, ws_bytes = workspace.data_ptr(), need.value
    _hg._check(_lib.engram_paged_attention(at, ws, ws_bytes or 0, _hg._stream(stream)), "engram_paged_attention")
    return (out, lse) if return_lse else out
