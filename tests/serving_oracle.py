"""Plain 64-bit forms of the serving operators (CPU), and the tolerances of their comparisons.

A rounding to a 16-bit type is off by at most half a step, eps / 2 of the value; fp32 steps count 2^-24 each.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def normed(x, weight, eps):
    x = x.double()
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def rotated(x, positions, inv_freq, interleaved):
    """[T, H, D] float64 -> (rotated, |a| + |b| of each element's pair): element by element from the definition."""
    x = x.double()
    size = x.abs()
    if inv_freq is None:
        return x, size
    half = inv_freq.numel()
    out, size = x.clone(), size.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = positions.double() * inv_freq[i].double()
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, size


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """(value, fp32 error bound).  The norm's sum, root, reciprocal and two products are within 24 fp32 steps of the
    element, the rotation within 8 of the pair (cos and sin 2 each, two products, one sum, each term)."""
    y = normed(x, weight, eps)
    out, size = rotated(y, positions, inv_freq, interleaved)
    return out, 32 * U32 * size


def rounding_bound(value, fp32_bound, dtype):
    """Half a step of the rounded value (below the normal range: of the smallest normal), and what fp32 was off."""
    tiny = torch.finfo(dtype).tiny
    return half_step(dtype) * (value.abs() + fp32_bound).clamp(min=tiny) + fp32_bound


def attention(q, k_cache, v_cache, table, kv_len, cu_q, scale, window, k_scale=None, v_scale=None):
    """(out, lse, bound of out from fp32 and P in about 16 bits, bound of lse), request by request in float64.

    Pages outside of the pool count as unseen.  A score is off by (D + 8) fp32 steps of scale * sum |q k|, which moves a
    weight by as much; a sum of n terms adds n / 64 (each lane adds its own) and is divided out."""
    T, Hq, D = q.shape
    n_pages, H, page, _ = k_cache.shape
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    move = torch.zeros((T, Hq), dtype=torch.float64)
    mass = torch.zeros((T, Hq, D), dtype=torch.float64)
    q = q.double()

    def rows(cache, scales, ids, place):
        r = cache[ids, :, place]
        if scales is not None:
            return r.view(torch.float8_e4m3fn).double() * scales[ids, :, place].double()[..., None]
        return r.double()

    for b in range(len(kv_len)):
        t0, t1 = int(cu_q[b]), int(cu_q[b + 1])
        length = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        for t in range(t0, t1):
            p = length - (t1 - t0) + (t - t0)
            lo = max(0, p - window + 1) if window else 0
            if p < 0 or lo > p:
                continue
            key = torch.arange(lo, p + 1)
            ids = table[b].long()[key // page]
            real = (ids >= 0) & (ids < n_pages)
            key, ids = key[real], ids[real]
            if key.numel() == 0:
                continue
            kk, vv = rows(k_cache, k_scale, ids, key % page), rows(v_cache, v_scale, ids, key % page)
            for h in range(H):
                qq = q[t, h * G:(h + 1) * G]
                s = qq @ kk[:, h].T * scale
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - z[:, None])
                sl = slice(h * G, (h + 1) * G)
                lse[t, sl] = z
                out[t, sl] = w @ vv[:, h]
                mass[t, sl] = w @ vv[:, h].abs()
                size = (qq.abs() @ kk[:, h].abs().T * abs(scale)).amax(-1)
                move[t, sl] = (D + 8) * U32 * size + (key.numel() / 64 + 8) * U32
    return out, lse, mass, move


def attention_bounds(out, lse, mass, move, dtype, p_half_step):
    """Elementwise bounds: the output's rounding, weights moved by `move` (twice: numerator and sum), and each weight's
    own rounding to p_half_step of its value."""
    fp = mass * (2 * move[..., None] + p_half_step)
    return rounding_bound(out, fp, dtype), move + 8 * U32 * (1 + lse.abs().nan_to_num(posinf=0.0))
