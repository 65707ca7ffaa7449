"""Plain 64-bit forms of the calls of a drafting step (CPU): page tables and slots, appends to pages with one scale each,
verification of drafts."""
from __future__ import annotations

import math

import torch

import serving_oracle as so

LARGEST = {"e4m3": 448.0, "int8": 127.0}


def page_tables(lengths, new, table, held, stack, n_free, page, n_tok):
    """Request by request: a dict of all outputs, updated state among them (numbers and lists of Python)."""
    n, width = len(lengths), len(table[0]) if len(table) else 0
    length, new = [max(x, 0) for x in lengths], [max(x, 0) for x in new]
    table, stack = [list(r) for r in table], list(stack)
    held_in = [min(max(h, 0), width) for h in held]
    held_out = list(held)
    n_free = min(max(n_free, 0), len(stack))
    need = [-(-(a + m) // page) for a, m in zip(length, new)]
    cu, fits = [0], []
    for b in range(n):
        end = sum(new[:b + 1])
        cu.append(min(end, n_tok))
        fits.append((end <= n_tok or new[b] == 0) and need[b] <= width and length[b] + new[b] <= 2 ** 31 - 4096)
    back = [table[b][p] for b in range(n) if fits[b] for p in range(need[b], held_in[b])]
    pool = back + [stack[i] for i in range(n_free - 1, -1, -1)]
    wanted = dealt = short = 0
    out = {"slots": [-1] * n_tok, "positions": [0] * n_tok, "cu_q": cu, "kv_len": []}
    for b in range(n):
        take = max(need[b] - held_in[b], 0) if fits[b] else 0
        wanted += take
        served = fits[b] and (take == 0 or wanted <= len(pool))
        if served:
            for p in range(take):
                table[b][held_in[b] + p] = pool[dealt]
                dealt += 1
            held_out[b] = need[b]
            for i in range(new[b]):
                p = length[b] + i
                out["slots"][cu[b] + i] = table[b][p // page] * page + p % page
                out["positions"][cu[b] + i] = p
        out["kv_len"].append(length[b] + new[b] if served else 0)
        short += not served
    left = n_free - max(dealt - len(back), 0)
    for x in back[dealt:]:
        if left < len(stack):
            stack[left] = x
            left += 1
    return dict(out, n_short=[short], table=table, held=held_out, free=stack, n_free=[left])


def power_of_two(x):
    """The least power of two, 2^-126 at least, that is not below x (float64; 0 for 0)."""
    m, e = torch.frexp(x.double())
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    return torch.where(x > 0, torch.exp2(e.double()), 0.0)


def values(codes, kind):
    return codes.double() if kind == "int8" else codes.view(torch.float8_e4m3fn).double()


def nearest(x, kind):
    """The value of the code nearest to x, ties to even (float64)."""
    if kind == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def append(x, fp, cache, scale, table, kv_len, cu, kind):
    """Rows x [T, H, D] (float64, fp32 computed them within fp) appended to a cache: (values of all codes, scales, bound of
    codes * scale, the least and most that each scale may be), from the cache as it is before."""
    n_pages, H, page, D = cache.shape
    held, scale = values(cache, kind), scale.double().clone()
    low, high = scale.clone(), scale.clone()
    bound = torch.zeros_like(held)
    for b in range(len(kv_len)):
        n = int(cu[b + 1] - cu[b])
        length = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        for key0 in range(max(length - n, 0) // page * page, length, page):
            p = int(table[b, key0 // page])
            a, e = max(length - n, 0, key0), min(length, key0 + page)
            if a >= e or not 0 <= p < n_pages:
                continue
            t = int(cu[b]) + a - (length - n)
            rows, off = x[t:t + e - a].transpose(0, 1), fp[t:t + e - a].transpose(0, 1)  # [H, n, D]
            r = a - key0
            size = rows.abs()
            some = [power_of_two(y.amax((1, 2)) / LARGEST[kind]) for y in (size, (size - off).clamp(min=0), size + off)]
            bad = ~torch.isfinite(rows).all(-1).all(-1)
            before = scale[p].clone() if r else torch.zeros(H, dtype=torch.float64)
            now, low[p], high[p] = (torch.where(bad | before.isnan(), math.nan, torch.maximum(y, before)) for y in some)
            unit = torch.where(now > 0, now, 1.0)[:, None, None]
            if r:
                ratio = (before[:, None, None] / unit)
                held[p, :, :r] = torch.where((now > before)[:, None, None], nearest(held[p, :, :r] * ratio, kind), held[p, :, :r])
            held[p, :, r:e - key0] = nearest(rows / unit, kind)
            scale[p] = now
            # what fp32 moved may round to the next code: half a step of a code more on either side (its own step; steps of
            # 2^-9 below 2^-6), and what it moved
            half = (unit / 2 if kind == "int8" else (rows.abs() + off) * 2.0 ** -4 + unit * 2.0 ** -10)
            bound[p, :, r:e - key0] = torch.where(off > 0, 2 * half + off, 0.0)
    return held, scale, bound, low, high


def verify(target, draft, uniform, last, q, cu):
    """Request by request in float64: (tokens, accepted)."""
    tokens, accepted = [], []
    V = target.shape[1]
    for b in range(len(cu) - 1):
        a, n, w = 0, int(cu[b + 1] - cu[b]), None
        for i in range(n):
            t = int(cu[b]) + i
            p, d = target[t + b].double(), int(draft[t])
            real = 0 <= d < V
            if q is None:
                qi = torch.zeros(V, dtype=torch.float64)
                if real:
                    qi[d] = 1.0
            else:
                qi = q[t].double()
            pd = float(p[d]) if real else 0.0
            qd = float(qi[d]) if real else 1.0
            if float(uniform[t]) * qd < pd:
                a += 1
                continue
            w = torch.where(p > qi, p - qi, 0.0).nan_to_num(nan=0.0, posinf=math.inf)
            if q is None and real:
                w = torch.where(p > 0, p, 0.0)
                w[d] = 0.0
            if not float(w.sum()) > 0:
                w = None
            break
        row = target[int(cu[b]) + a + b].double()
        if w is None:
            w = torch.where(row > 0, row, 0.0)
        total = float(w.sum())
        if not (0 < total < math.inf):
            word = -1
        else:
            upto = w.cumsum(0)
            v = float(last[b])
            pick = (upto > (v if v > 0 else 0.0) * float(upto[-1])) & (w > 0)
            word = int(pick.int().argmax()) if pick.any() else int((w > 0).nonzero()[-1])
        tokens += [int(x) for x in draft[int(cu[b]):int(cu[b]) + a]] + [word] + [-1] * (n - a)
        accepted.append(a)
    return tokens, accepted


