"""Serving operators next to the lookup: head norm + rotation, paged cache appends, paged attention, and between the steps
page tables, slots and the verification of drafts.

Argument marshalling only, as in the package's own module; the C ABI is in
include/engram.h.  A cache is a pair of device tensors [n_pages, n_kv_heads,
page_size, head_dim] that the caller owns: bfloat16 or float16, or codes with
float32 scales for K and V: FP8 E4M3 (uint8 or float8_e4m3fn) with scales
[n_pages, n_kv_heads, page_size] or [n_pages, n_kv_heads], int8 with the latter.

    q, _ = qk_norm_rope(q, None, positions, inv_freq, q_weight=wq)       # engram_qk_norm_rope
    kv_append(k, v, k_cache, v_cache, slots, positions=positions, inv_freq=inv_freq, k_weight=wk)  # engram_kv_append
    out = paged_attention(q, k_cache, v_cache, block_table, kv_len)       # engram_paged_attention

A batch that goes on by itself, with a cache of one scale for each page and head:

    slots, positions, cu_q, kv_len, n_short = page_tables(lengths, new, block_table, held, free_pages, n_free, page_size, n_tok)
    kv_append_pages(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, cu_q, ...)  # engram_kv_append_pages
    tokens, n_accepted = verify_draft(target, draft, uniform, last_uniform, draft_probs)  # engram_verify_draft

attention_example.py runs the first together, next to the lookup, drafting_example.py all of them.

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

BF16, F16, E4M3, E4M3_PAGE, I8_PAGE, F32 = 0, 1, 2, 4, 5, 6


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


class AppendPagesDesc(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(KvCacheDesc)), ("k", _VP), ("v", _VP), ("k_weight", _VP), ("positions", _VP),
                ("inv_freq", _VP), ("block_table", _VP), ("kv_len", _VP), ("cu_q", _VP), ("n_seq", _I64), ("n_tok", _I64),
                ("max_q_len", _I64), ("table_width", _I64), ("table_stride", _I64), ("k_token_stride", _I64),
                ("k_head_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64), ("rotary_dim", _U32),
                ("interleaved", _U32), ("type", _U32), ("eps", _F32), ("reserved0", _U32)]


class PageTablesDesc(ctypes.Structure):
    _fields_ = [("lengths", _VP), ("new_tokens", _VP), ("block_table", _VP), ("held", _VP), ("free_pages", _VP),
                ("n_free", _VP), ("slots", _VP), ("positions", _VP), ("cu_q", _VP), ("kv_len", _VP), ("n_short", _VP),
                ("n_seq", _I64), ("n_tok", _I64), ("table_width", _I64), ("table_stride", _I64), ("n_pages", _I64),
                ("page_size", _U32), ("reserved0", _U32)]


class VerifyDraftDesc(ctypes.Structure):
    _fields_ = [("target", _VP), ("draft_probs", _VP), ("draft", _VP), ("uniform", _VP), ("last_uniform", _VP),
                ("cu_draft", _VP), ("tokens", _VP), ("n_accepted", _VP), ("n_seq", _I64), ("n_draft", _I64), ("vocab", _I64),
                ("target_stride", _I64), ("draft_stride", _I64), ("type", _U32), ("reserved0", _U32)]


_SIZE_P = ctypes.POINTER(ctypes.c_size_t)
_lib = _hg.lib()
for _name, _args in {"engram_qk_norm_rope": [_VP, _VP], "engram_kv_append": [_VP, _VP], "engram_kv_append_pages": [_VP, _VP],
                     "engram_page_tables_workspace": [_VP, _SIZE_P], "engram_page_tables": [_VP, _VP, ctypes.c_size_t, _VP],
                     "engram_verify_draft_workspace": [_VP, _SIZE_P], "engram_verify_draft": [_VP, _VP, ctypes.c_size_t, _VP],
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


def kv_append_pages(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor, cu_q: torch.Tensor | None = None,
                    max_q_len: int | None = None, positions: torch.Tensor | None = None,
                    inv_freq: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                    interleaved: bool = False, stream=None) -> None:
    """kv_append for a cache of codes (e4m3, int8) with one scale for each page and head, ``k_scale`` and ``v_scale`` float32
    [n_pages, n_kv_heads]: request b's new tokens cu_q[b] .. cu_q[b+1]-1 (None: equally many each) are the last of its
    kv_len[b] keys, on the pages block_table[b] (engram_kv_append_pages).

    A page's scale is a power of two and only grows while the page fills; codes held are rounded again when it does.  A page
    belongs to one request.  ``max_q_len`` bounds the tokens of a request where it is known: single tokens take a smaller
    kernel, and what is past it may be left out."""
    args = (k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, cu_q, max_q_len, positions, inv_freq, k_weight, eps,
            interleaved)
    if stream is None:
        return _serving.kv_append_pages(*args)
    with _on(stream, k):
        return _serving.kv_append_pages(*args)


def page_tables(lengths: torch.Tensor, new_tokens: torch.Tensor | None, block_table: torch.Tensor, held: torch.Tensor,
                free_pages: torch.Tensor, n_free: torch.Tensor, page_size: int, n_tok: int,
                workspace: torch.Tensor | None = None, stream=None):
    """Make every request hold the pages that its length needs, and place its new tokens (engram_page_tables): (slots int64
    [n_tok], positions int32 [n_tok], cu_q int32 [n_seq + 1], kv_len int32 [n_seq], n_short int32 [1]).

    Request b has ``lengths[b]`` keys (int32 [n_seq]) and gets ``new_tokens[b]`` more (None: n_tok / n_seq each), and holds
    the first ``held[b]`` pages of block_table[b] (int32 [n_seq, width]).  Pages past its need come back, those missing are
    taken from what came back and then from the top of the stack ``free_pages`` [n_pages], of which ``n_free`` [1] count;
    block_table, held, free_pages and n_free are brought up to date.  A request that cannot be served (n_short of them) keeps
    what it holds; its tokens get slot -1 and its kv_len is 0, so that it is appended to and attended by nothing.  A request
    of length 0 without new tokens gives back all that it holds.  ``n_tok`` is the batch's size; tokens past the requests'
    own get slot -1.  ``workspace``: uint8 of page_tables_workspace bytes, 256-byte aligned; allocated if not given."""
    args = (lengths, new_tokens, block_table, held, free_pages, n_free, page_size, n_tok, workspace, False)
    if stream is None:
        return _serving.page_tables(*args)
    with _on(stream, block_table):
        return _serving.page_tables(*args)


def page_tables_workspace(lengths: torch.Tensor, new_tokens: torch.Tensor | None, block_table: torch.Tensor,
                          held: torch.Tensor, free_pages: torch.Tensor, n_free: torch.Tensor, page_size: int,
                          n_tok: int) -> int:
    """Bytes of the workspace that page_tables needs with these arguments; it goes by their shapes and ``n_tok`` alone
    (engram_page_tables_workspace)."""
    return _serving.page_tables(lengths, new_tokens, block_table, held, free_pages, n_free, page_size, n_tok, None, True)


def verify_draft(target: torch.Tensor, draft: torch.Tensor, uniform: torch.Tensor, last_uniform: torch.Tensor,
                 draft_probs: torch.Tensor | None = None, cu_draft: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """Keep drafted tokens by the target's probabilities and draw the token after them (engram_verify_draft): (tokens int32
    [n_draft + n_seq], n_accepted int32 [n_seq]).

    Request b has the drafts cu_draft[b] .. cu_draft[b+1]-1 of ``draft`` int32 [n_draft] (None: equally many each) and one
    row of ``target`` [n_draft + n_seq, vocab] (float32, bfloat16 or float16) more than drafts, from cu_draft[b] + b on, as
    its tokens of ``tokens``: those accepted, the one after, then -1.  ``draft_probs`` [n_draft, vocab] are the
    probabilities that each draft was drawn from (None: it was certain).  ``uniform`` float32 [n_draft] and ``last_uniform``
    float32 [n_seq] are random numbers of [0, 1).  The tokens that come out are distributed as the target's own.
    ``workspace``: uint8 of verify_draft_workspace bytes, 256-byte aligned; allocated if not given."""
    args = (target, draft, uniform, last_uniform, draft_probs, cu_draft, workspace, False)
    if stream is None:
        return _serving.verify_draft(*args)
    with _on(stream, target):
        return _serving.verify_draft(*args)


def verify_draft_workspace(target: torch.Tensor, draft: torch.Tensor, uniform: torch.Tensor, last_uniform: torch.Tensor,
                           draft_probs: torch.Tensor | None = None, cu_draft: torch.Tensor | None = None) -> int:
    """Bytes of the workspace that verify_draft needs with these arguments; it goes by their shapes alone
    (engram_verify_draft_workspace)."""
    return _serving.verify_draft(target, draft, uniform, last_uniform, draft_probs, cu_draft, None, True)


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
