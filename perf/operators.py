"""The serving operators around the memory lookup, case by case: what one call takes, its plain form and its work.

Three operators carry a request's new tokens from the projections of an attention layer to its output, next to the
n-gram memory that the same tokens read:

* norm_rope: RMS norm of every query and key head and the rotation by position, in one pass;
* append:    new keys (normed and rotated on the way) and values into a paged cache, in bf16, fp16 or e4m3;
* attention: new tokens (one a request, or a chunk of a prompt) over the paged cache.

`run` computes the plain form with elementary torch operations where `own` is false, and calls the library where it is
true.  A cache is a pair of tensors [n_pages, kv_heads, page, dim]; an e4m3 cache holds codes and one fp32 scale for
each (page, head, slot).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm_rope(name, tokens, q_heads, kv_heads, dim, rotary, interleaved, dtype, first):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "dtype": dtype, "first": first}


def _append(name, tokens, kv_heads, dim, rotary, interleaved, norm, page, dtype, e4m3, first):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "norm": norm, "page": page, "dtype": dtype, "e4m3": e4m3, "first": first}


def _attention(name, seqs, new, context, q_heads, kv_heads, dim, page, window, dtype, e4m3, ragged, lse):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "context": context, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "dtype": dtype, "e4m3": e4m3,
            "ragged": ragged, "lse": lse}


def listed():
    return [
        # a single request's next token: what the call costs when there is nothing to do
        _norm_rope("norm rope, one token", 1, 32, 8, 128, 128, False, "bf16", 8191),
        # a whole prompt of the prefill workload
        _norm_rope("norm rope, prompt of 32768", 32768, 32, 8, 128, 128, False, "bf16", 0),
        # a small model with a partial, interleaved rotation, far into its context
        _norm_rope("norm rope, odd prompt", 1531, 14, 2, 64, 32, True, "fp16", 500000),
        # one decode step of the 64-request workload
        _append("append, 64 requests", 64, 8, 128, 128, False, True, 16, "bf16", False, 4096),
        # a whole prompt into the cache
        _append("append, prompt of 32768", 32768, 8, 128, 128, False, True, 16, "bf16", False, 0),
        # a prompt's odd tail into a cache of half the bytes
        _append("append, odd prompt, e4m3", 8191, 4, 128, 64, False, False, 32, "bf16", True, 100000),
        # one request with a short context: latency
        _attention("attention, one request", 1, 1, 512, 32, 8, 128, 16, 0, "bf16", False, False, False),
        # one decode step of 64 requests with contexts of up to 8,192 tokens
        _attention("attention, 64 requests", 64, 1, 8192, 32, 8, 128, 16, 0, "bf16", False, True, False),
        # the same over an e4m3 cache
        _attention("attention, 64 requests, e4m3", 64, 1, 8192, 32, 8, 128, 32, 0, "bf16", True, True, False),
        # one request at the full context of 131,072 tokens: the work has to be split over the context
        _attention("attention, far request", 1, 1, 131072, 32, 8, 128, 16, 0, "bf16", False, False, True),
        # a chunk of a long prompt over what the cache already holds
        _attention("attention, chunk of 2048", 1, 2048, 32768, 32, 8, 128, 16, 0, "bf16", False, False, False),
        # chunks and single tokens of many requests in one call, small heads, seven queries to a key, a window
        _attention("attention, mixed batch", 24, 512, 8192, 14, 2, 64, 16, 1024, "fp16", False, True, True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    rotary = rng.choice([16, dim // 2, dim])
    first = _spread(rng, 1, 1000000) - 1
    if op == "norm_rope":
        tokens = _spread(rng, 1, max(1, min(32768, 32768 * 40 * 128 // ((group + 1) * kv_heads * dim))))
        c = _norm_rope("", tokens, kv_heads * group, kv_heads, dim, rotary, rng.random() < 0.5, dtype, first)
    elif op == "append":
        tokens = _spread(rng, 1, max(1, min(32768, 32768 * 8 * 128 // (kv_heads * dim))))
        c = _append("", tokens, kv_heads, dim, rotary, rng.random() < 0.5, rng.random() < 0.5, page, dtype,
                    rng.random() < 0.4, first)
    else:
        window = rng.choice([0, 0, 0, 128, _spread(rng, 1, 8192)])
        e4m3 = rng.random() < 0.4
        if rng.random() < 0.5:  # a decode step
            seqs, new = _spread(rng, 1, 128), 1
            most = 64 * 8192 * 8 * 128 // (seqs * kv_heads * dim)
            context = _spread(rng, 1, max(1, min(131072, most)))
        else:  # chunks, some with single tokens among them
            seqs, new = _spread(rng, 1, 16), _spread(rng, 2, 2048)
            most = 2048 * 32768 * 32 * 128 // (4 * seqs * new * kv_heads * group * dim)
            context = _spread(rng, new, max(new, min(32768, most)))
        c = _attention("", seqs, new, context, kv_heads * group, kv_heads, dim, page, window, dtype, e4m3,
                       rng.random() < 0.6, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of every request: the case alone says them."""
    rng = random.Random("%(seqs)d %(new)d %(context)d" % c)
    new, kv = [], []
    for b in range(c["seqs"]):
        if not c["ragged"] or b == 0:
            new.append(c["new"])
            kv.append(max(c["context"], c["new"]))
        else:
            n = 1 if c["new"] == 1 or rng.random() < 0.3 else rng.randint(0, c["new"])
            new.append(n)
            kv.append(rng.randint(max(n, 1), max(c["context"], n, 1)))
    return new, kv


def work(c):
    size = 2
    if c["op"] == "norm_rope":
        n = c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * n * size + 4 * c["tokens"] + 2 * c["dim"] * size + 4 * c["rotary"], "flops": 7 * n}
    if c["op"] == "append":
        n = c["tokens"] * c["kv_heads"] * c["dim"]
        out = 2 * n + 8 * c["tokens"] * c["kv_heads"] if c["e4m3"] else 2 * n * size
        return {"bytes": 2 * n * size + out + 12 * c["tokens"] + 4 * c["rotary"], "flops": 7 * n}
    new, kv = _lengths(c)
    pairs = tokens = 0
    for n, k in zip(new, kv):
        if n == 0:
            continue
        w = c["window"] or k
        pairs += sum(min(k - n + 1 + j, w) for j in range(n))
        tokens += min(k, w + n - 1)
    row = c["dim"] * (1 if c["e4m3"] else size) + (4 if c["e4m3"] else 0)
    rows = sum(new) * c["q_heads"]
    return {"bytes": 2 * rows * c["dim"] * size + 2 * tokens * c["kv_heads"] * row + rows * (4 if c["lse"] else 0)
            + 8 * c["seqs"] + sum(-(-k // c["page"]) for k in kv) * 4,
            "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = np.random.default_rng(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(t)

    s = {"case": c, "eps": 1e-6}
    D = c["dim"]
    if c["op"] in ("norm_rope", "append"):
        # a projection's output: queries, keys and values of a token side by side; keys and values grow with the
        # channel as trained ones do
        T, H = c["tokens"], c["kv_heads"]
        Hq = c.get("q_heads", H)
        qkv = normal(T, Hq + 2 * H, D, std=2.0)
        qkv *= (0.25 + 1.5 * torch.rand((Hq + 2 * H, D), generator=g, device=dev)).to(t)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["positions"] = torch.arange(c["first"], c["first"] + T, dtype=torch.int32, device=dev)
        R = c["rotary"]
        base = 1e4 if seed % 2 else 1e6
        s["inv_freq"] = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
        s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(t)
        s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(t)
        if c["op"] == "append":
            page = c["page"]
            pages = -(-T // page) + 2
            order = host.permutation(pages)  # where the pool had room
            at = np.arange(T) + int(host.integers(0, page))
            slots = order[at // page] * page + at % page
            slots[host.random(T) < 0.02] = -1  # padding of a batch
            s["slots"] = torch.from_numpy(slots.astype(np.int64)).to(dev)
            shape = (pages, H, page, D)
            if c["e4m3"]:
                s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2))
                s["k_scale"], s["v_scale"] = (torch.zeros(shape[:3], device=dev) for _ in range(2))
            else:
                s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=t, device=dev) for _ in range(2))
            if not c["norm"]:
                s["k_weight"] = None
        return s
    new, kv = _lengths(c)
    H, page = c["kv_heads"], c["page"]
    need = [-(-k // page) for k in kv]
    pages = sum(need) + 3
    order = host.permutation(pages)
    table = np.zeros((c["seqs"], max(need)), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = torch.from_numpy(table).to(dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["max_q_len"] = max(new)
    s["cu_q"] = None
    if len(set(new)) > 1:
        s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
    s["q"] = normal(sum(new), c["q_heads"], D, std=1.5)
    shape = (pages, H, page, D)
    if c["e4m3"]:
        for x, std in (("k", 1.0), ("v", 1.0)):
            r = torch.randn(shape, generator=g, device=dev) * std
            scale = r.abs().amax(-1) / E4M3_MAX
            s[x + "_cache"] = (r / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s[x + "_scale"] = scale
    else:
        s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
        s["k_scale"] = s["v_scale"] = None
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _rotated(x, weight, s):
    """RMS norm (where there is a weight) and rotation of [T, H, D] in 32 bits; angles in 64."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    R = c["rotary"]
    head, rest = x[..., :R], x[..., R:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., :R // 2], head[..., R // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([head, rest], -1)


def _plain_append(s):
    c = s["case"]
    k, v = _rotated(s["k"], s["k_weight"], s), s["v"].float()
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][keep]
    page, at = slot // c["page"], slot % c["page"]
    for x, name in ((k[keep], "k"), (v[keep], "v")):
        if c["e4m3"]:
            scale = x.abs().amax(-1) / E4M3_MAX
            s[name + "_scale"][page, :, at] = scale
            x = (x / torch.where(scale > 0, scale, 1.0)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_cache"][page, :, at] = x.to(s[name + "_cache"].dtype)


def _plain_attention(s):
    c = s["case"]
    table, page, H, D = s["table"].long(), c["page"], c["kv_heads"], c["dim"]
    B, L = table.shape[0], table.shape[1] * page
    G = c["q_heads"] // H

    def cached(x):
        r = s[x + "_cache"][table]
        r = r.view(torch.float8_e4m3fn).float() * s[x + "_scale"][table][..., None] if c["e4m3"] else r.float()
        return r.transpose(1, 2).reshape(B, H, L, D)

    k, v = cached("k"), cached("v")
    T, N = s["q"].shape[0], s["max_q_len"]
    dev = s["q"].device
    if s["cu_q"] is None:
        start = torch.arange(B, device=dev) * N
        count = torch.full((B,), N, device=dev)
    else:
        start, count = s["cu_q"][:-1].long(), s["cu_q"].diff().long()
    j = torch.arange(N, device=dev)
    q = s["q"].float()[(start[:, None] + j).clamp(max=T - 1)]  # [B, N, Hq, D]
    q = q.reshape(B, N, H, G, D).transpose(1, 2).reshape(B, H, N * G, D)
    score = torch.matmul(q * s["scale"], k.transpose(2, 3).contiguous())
    last = s["kv_len"].long()[:, None] - count[:, None] + j  # the newest key that each query may see
    at = torch.arange(L, device=dev)
    hidden = at > last[..., None]
    if c["window"]:
        hidden |= at <= last[..., None] - c["window"]
    score.view(B, H, N, G, L).masked_fill_(hidden[:, None, :, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    score.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v) / torch.where(total > 0, total, 1.0)
    lse = (most + total.log()).reshape(B, H, N, G).transpose(1, 2).reshape(B, N, H * G)
    out = out.reshape(B, H, N, G, D).transpose(1, 2).reshape(B, N, H * G, D)
    tok = torch.arange(T, device=dev)
    b = torch.searchsorted(start + count, tok, right=True)
    out = out[b, tok - start[b]].to(s["q"].dtype)
    return (out, lse[b, tok - start[b]]) if c["lse"] else out


def run(s):
    c = s["case"]
    if own:
        import hashed_gram_memory_amd as hg

        if c["op"] == "norm_rope":
            return hg.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=s["eps"], interleaved=c["interleaved"])
        if c["op"] == "append":
            hg.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], positions=s["positions"],
                         inv_freq=s["inv_freq"], k_weight=s["k_weight"], eps=s["eps"], interleaved=c["interleaved"],
                         k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        else:
            return hg.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], cu_q=s["cu_q"],
                                      max_q_len=s["max_q_len"], scale=s["scale"], window=c["window"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=c["lse"])
    elif c["op"] == "norm_rope":
        return tuple(_rotated(s[x], s[x + "_weight"], s).to(s["q"].dtype) for x in ("q", "k"))
    elif c["op"] == "append":
        _plain_append(s)
    else:
        return _plain_attention(s)
    if c["e4m3"]:
        return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
                "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return {"k": s["k_cache"], "v": s["v_cache"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, weight, s):
    """The norm and the rotation of [T, H, D], each pair as a complex number."""
    c, x = s["case"], x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * weight.double()
    R = c["rotary"]
    pair = x[..., :R].unflatten(-1, (R // 2, 2) if c["interleaved"] else (2, R // 2))
    if not c["interleaved"]:
        pair = pair.transpose(-1, -2)
    turn = torch.exp(1j * (s["positions"].double().unsqueeze(-1) * s["inv_freq"]))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn.unsqueeze(1))
    if not c["interleaved"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., R:]), dim=-1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        return _turned(s["q"], s["q_weight"], s), _turned(s["k"], s["k_weight"], s)
    if c["op"] == "append":
        held, H, D, page = {}, c["kv_heads"], c["dim"], c["page"]
        real = torch.nonzero(s["slots"] != -1).flatten()
        for name, x in (("k", _turned(s["k"], s["k_weight"], s)), ("v", s["v"].double())):
            flat = torch.zeros((s[name + "_cache"].shape[0] * page, H, D), dtype=torch.float64, device=x.device)
            x = x[real]
            if c["e4m3"]:
                step = x.abs().max(-1).values / 448
                scales = torch.zeros(flat.shape[:2], dtype=torch.float64, device=x.device)
                scales[s["slots"][real]] = step
                held[name + "_scale"] = scales.reshape(-1, page, H).transpose(1, 2).contiguous()
                x = torch.where(step[..., None] > 0, x / step[..., None], torch.zeros_like(x))
                # the nearest e4m3 value, ties to even: 3 bits below the leading one, steps of 2^-9 at least
                grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                x = torch.round(x / grid) * grid
            flat[s["slots"][real]] = x
            held[name] = flat.reshape(-1, page, H, D).transpose(1, 2).contiguous()
        return held
    new, kv = _lengths(c)
    H, G, D = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
    outs, lses = [], []
    at = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        if n == 0:
            continue
        low = max(0, length - n + 1 - c["window"]) if c["window"] else 0
        key = torch.arange(low, length, device=s["q"].device)
        ids = s["table"][b].long()[key // c["page"]]
        newest = torch.arange(length - n, length, device=key.device)
        seen = key <= newest[:, None]
        if c["window"]:
            seen &= newest[:, None] - key < c["window"]
        heads, logs = [], []
        for h in range(H):
            kk, vv = (s[x + "_cache"][ids, h, key % c["page"]] for x in "kv")
            if c["e4m3"]:
                kk, vv = (r.view(torch.float8_e4m3fn).double() * s[x + "_scale"][ids, h, key % c["page"]].double()[:, None]
                          for r, x in ((kk, "k"), (vv, "v")))
            kk, vv = kk.double(), vv.double()
            for i in range(G):
                z = s["q"][at:at + n, h * G + i].double() @ kk.t().contiguous() * s["scale"]
                z = torch.where(seen, z, -math.inf)
                log = torch.logsumexp(z, -1)
                heads.append(torch.exp(z - log[:, None]) @ vv)
                logs.append(log)
        outs.append(torch.stack(heads, 1))
        lses.append(torch.stack(logs, 1))
        at += n
    return (torch.cat(outs), torch.cat(lses)) if c["lse"] else torch.cat(outs)
