"""A step of speculative decoding over a paged cache of 8 bits, case by case: what one call takes, its plain form, its work.

Operators that let a batch of requests go on from step to step on the GPU, next to the n-gram memory that reads the same
tokens and the attention layer around it:

* tables:    the pages of every request made to fit its length (free pages dealt, surplus ones given back), and the
             slots, positions and offsets of the step's tokens;
* append:    new keys (normed and rotated on the way) and values into a cache of 8 bits, e4m3 or int8, with one scale for
             each page and head;
* attention: new tokens (one a request, drafted ones, or a chunk of a prompt) over such a cache;
* verify:    drafted tokens kept or refused by the target's probabilities and given random numbers, and the token after.

`run` computes the plain form with elementary torch operations where `own` is false, and calls the library where it is
true.  A cache is a pair of tensors [n_pages, kv_heads, page, dim] of codes with scales [n_pages, kv_heads].
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LARGEST = {"e4m3": 448.0, "int8": 127.0}  # code of each kind


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tables(name, seqs, new, context, page, ragged, scarce):
    """`new` tokens at most for each of `seqs` requests of up to `context` keys; `scarce`: too few free pages for all."""
    return {"name": name, "op": "tables", "seqs": seqs, "new": new, "context": context, "page": page, "ragged": ragged,
            "scarce": scarce}


def _append(name, seqs, new, context, kv_heads, dim, rotary, interleaved, norm, page, dtype, kind, ragged):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "context": context, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "norm": norm, "page": page, "dtype": dtype, "kind": kind,
            "ragged": ragged}


def _attention(name, seqs, new, context, q_heads, kv_heads, dim, page, window, dtype, kind, ragged, lse):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "context": context, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "dtype": dtype, "kind": kind,
            "ragged": ragged, "lse": lse}


def _verify(name, seqs, drafts, vocab, dtype, ragged, given):
    """Up to `drafts` drafted tokens a request; `given`: their drafter's probabilities are there (else it was sure)."""
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab, "dtype": dtype,
            "ragged": ragged, "given": given}


def listed():
    return [
        # a decode step of 64 requests with five drafted tokens each: what the call costs when there is little to do
        _tables("tables, 64 requests", 64, 6, 8192, 16, False, False),
        # prompts of many requests dealt out at once, into a pool that does not hold them all
        _tables("tables, prompts", 512, 1024, 1024, 16, True, True),
        # one decode step of 64 requests
        _append("append, 64 requests, int8", 64, 1, 8192, 8, 128, 128, False, True, 16, "bf16", "int8", True),
        # a whole prompt of the prefill workload
        _append("append, prompt of 32768, e4m3", 1, 32768, 32768, 8, 128, 128, False, True, 64, "bf16", "e4m3", False),
        # odd tails of prompts, keys that were turned before
        _append("append, odd chunks, int8", 5, 1531, 100000, 4, 64, 0, False, False, 32, "fp16", "int8", True),
        # one decode step of 64 requests with contexts of up to 8,192 tokens
        _attention("attention, 64 requests, int8", 64, 1, 8192, 32, 8, 128, 16, 0, "bf16", "int8", True, False),
        # five drafted tokens of each of 16 requests checked in one pass: 24 rows to a key's head
        _attention("attention, drafts, e4m3", 16, 6, 8192, 32, 8, 128, 32, 0, "bf16", "e4m3", True, False),
        # one request at the full context of 131,072 tokens: the work has to be split over the context
        _attention("attention, far request, int8", 1, 1, 131072, 32, 8, 128, 64, 0, "bf16", "int8", False, True),
        # a chunk of a long prompt over what the cache already holds
        _attention("attention, chunk of 2048, int8", 1, 2048, 32768, 32, 8, 128, 16, 0, "bf16", "int8", False, False),
        # one request's drafts over a small vocabulary: latency
        _verify("verify, one request", 1, 5, 32768, "fp32", False, True),
        # one step of 64 requests
        _verify("verify, 64 requests", 64, 5, 129280, "fp32", False, True),
        # an odd vocabulary, some requests without a draft, in half the bytes
        _verify("verify, odd batch", 37, 7, 99091, "bf16", True, True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "verify", "verify"])
    page = rng.choice([8, 16, 32, 64, 128])
    ragged = rng.random() < 0.6
    dtype = rng.choice(["bf16", "fp16"])
    kind = rng.choice(["e4m3", "int8"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "tables":
        seqs = _spread(rng, 1, 1024)
        new = _spread(rng, 1, max(1, min(4096, 512 * 512 // seqs)))
        c = _tables("", seqs, new, _spread(rng, new, max(new, 32768)), page, ragged, rng.random() < 0.3)
    elif op == "append":
        norm = kind == "e4m3" and rng.random() < 0.5  # a key that arithmetic in 32 bits has moved may round to the next code
        rotary = rng.choice([16, dim // 2, dim]) if kind == "e4m3" else 0
        seqs = _spread(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, 32768 * 8 * 128 // (seqs * kv_heads * dim)))
        new = min(new, 32768)
        context = _spread(rng, new, max(new, min(131072, 131072 * 8 * 128 * 4 // (seqs * kv_heads * dim))))
        c = _append("", seqs, new, context, kv_heads, dim, rotary, rng.random() < 0.5, norm, page, dtype, kind, ragged)
    elif op == "attention":
        group = rng.choice([1, 2, 4, 5, 7, 8])
        window = rng.choice([0, 0, 0, 128, _spread(rng, 1, 8192)])
        if rng.random() < 0.6:  # a decode step, with drafts or without
            seqs, new = _spread(rng, 1, 128), rng.choice([1, 1, 2, 4, 6, 8])
            most = 64 * 8192 * 8 * 128 // (seqs * kv_heads * dim * new)
            context = _spread(rng, new, max(new, min(131072, most)))
        else:  # chunks, some with single tokens among them
            seqs, new = _spread(rng, 1, 16), _spread(rng, 9, 2048)
            most = 2048 * 32768 * 32 * 128 // (4 * seqs * new * kv_heads * group * dim)
            context = _spread(rng, new, max(new, min(32768, most)))
        c = _attention("", seqs, new, context, kv_heads * group, kv_heads, dim, page, window, dtype, kind, ragged,
                       rng.random() < 0.5)
    else:
        drafts = rng.choice([1, 2, 3, 4, 5, 7, 8])
        vocab = _spread(rng, 1000, 262144)
        seqs = _spread(rng, 1, max(1, min(256, 64 * 6 * 129280 // ((drafts + 1) * vocab))))
        c = _verify("", seqs, drafts, vocab, rng.choice(["fp32", "fp32", "bf16", "fp16"]), ragged, rng.random() < 0.7)
    del c["name"]
    return c


def _lengths(c):
    """New tokens and keys (the new ones among them) of every request: the case alone says them."""
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


def _drafts(c):
    """Drafted tokens of every request."""
    rng = random.Random("%(seqs)d %(drafts)d" % c)
    return [rng.randint(0, c["drafts"]) if c["ragged"] and b else c["drafts"] for b in range(c["seqs"])]


def work(c):
    if c["op"] == "tables":
        new, kv = _lengths(c)
        # a request: lengths, new tokens, pages held (in and out), keys, offset; a token: slot and position; a page: from
        # the pool to the table
        dealt = sum(-(-k // c["page"]) - -(-(k - n) // c["page"]) for n, k in zip(new, kv))
        return {"bytes": 24 * c["seqs"] + 12 * sum(new) + 8 * dealt, "flops": 4 * c["seqs"] + 4 * sum(new)}
    if c["op"] == "verify":
        k = _drafts(c)
        size = torch.empty((), dtype=TYPES[c["dtype"]]).element_size()
        # one row of the target's a request; of the drafter's where a draft is refused: with 7 of 10 kept, as here
        rows = len(k) + (sum(1 - 0.7 ** n for n in k) if c["given"] else 0)
        return {"bytes": int(rows * c["vocab"] * size) + 16 * sum(k) + 12 * len(k), "flops": int(2 * rows * c["vocab"])}
    new, kv = _lengths(c)
    D, H, page = c["dim"], c["kv_heads"], c["page"]
    if c["op"] == "append":
        n = sum(new) * H * D
        pages = sum(-(-k // page) - (k - m) // page for m, k in zip(new, kv) if m)
        return {"bytes": 2 * n * 2 + 2 * n + 8 * pages * H + 4 * sum(new) + 8 * c["seqs"] + 4 * pages + 4 * c["rotary"],
                "flops": 10 * n}
    pairs = tokens = 0
    for n, k in zip(new, kv):
        if n == 0:
            continue
        w = c["window"] or k
        pairs += sum(min(k - n + 1 + j, w) for j in range(n))
        tokens += min(k, w + n - 1)
    rows = sum(new) * c["q_heads"]
    return {"bytes": 4 * rows * D + 2 * tokens * H * D + 8 * (tokens // page) * H + rows * (4 if c["lse"] else 0)
            + 8 * c["seqs"] + sum(-(-k // page) for k in kv) * 4, "flops": 4 * pairs * c["q_heads"] * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pool(need, spare, host, width=None, others=0):
    """Pages in a random order: a table of `need[b]` of them each, and `spare` free ones (`others` are somebody else's)."""
    pages = sum(need) + spare + others
    order = host.permutation(pages).astype(np.int32)
    table = np.full((len(need), max(max(need), 1, width or 0)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:at + spare], pages


def _prepare_tables(c, s, host, dev):
    new, kv = _lengths(c)
    page = c["page"]
    need = [-(-k // page) for k in kv]
    # what each holds before the step; some hold pages of drafted tokens that were refused
    rng = random.Random("%(seqs)d %(context)d %(new)d" % c)
    held = [-(-(k - n) // page) + (rng.random() < 0.1) for n, k in zip(new, kv)]
    wanted = sum(max(n - h, 0) for n, h in zip(need, held))
    spare = max(wanted // 2, 1) if c["scarce"] else wanted + rng.randint(1, 100)
    table, free, pages = _pool(held, spare, host, max(need) + 1, 1000)
    stack = np.full(pages, -1, dtype=np.int32)  # with room for every page
    stack[:spare] = free
    to = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s["lengths"], s["new"] = to([k - n for n, k in zip(new, kv)]), to(new)
    s["table"], s["held"], s["free"], s["n_free"] = to(table), to(held), to(stack), to([spare])
    s["n_tok"] = -(-max(sum(new), 1) // 8) * 8  # a batch's size is often a round one


def _prepare_verify(c, s, g, host, dev):
    k = _drafts(c)
    N, B, V, t = sum(k), c["seqs"], c["vocab"], TYPES[c["dtype"]]
    cu = np.concatenate([[0], np.cumsum(k)])
    seq = np.repeat(np.arange(B), k)
    logits = 2.5 * torch.randn((N + B, V), generator=g, device=dev)
    # a word that the text before it suggests, more or less strongly
    word = torch.randint(0, V, (N + B, 1), generator=g, device=dev)
    logits.scatter_(1, word, logits.logsumexp(-1, keepdim=True) + 6 * torch.rand((N + B, 1), generator=g, device=dev) - 2)
    s["target"] = torch.softmax(logits, -1).to(t)
    rows = torch.from_numpy(np.arange(N) + seq).to(dev)
    # a drafter that agrees with most of the target
    q = torch.softmax(logits[rows] + 0.8 * torch.randn((N, V), generator=g, device=dev), -1)
    if not N:
        s["draft"] = torch.zeros(0, dtype=torch.int32, device=dev)
    elif c["given"]:
        s["draft"] = torch.multinomial(q, 1, generator=g)[:, 0].int()
    else:
        s["draft"] = q.argmax(-1).int()
    s["draft_probs"] = q.to(t) if c["given"] else None
    s["uniform"] = torch.rand(N, generator=g, device=dev)
    s["last_uniform"] = torch.rand(B, generator=g, device=dev)
    s["cu_draft"] = None if len(set(k)) == 1 else torch.from_numpy(cu.astype(np.int32)).to(dev)


def _power_of_two(x):
    """The least power of two that is not below x (0 for 0)."""
    m, e = torch.frexp(x)
    bits = (e.int() - (m == 0.5).int() + 127) << 23
    return torch.where(x > 0, bits.view(torch.float32), 0.0)


def _coded(x, kind):
    """x (in units of its scale) as codes."""
    return x.round().to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, kind):
    return codes.float() if kind == "int8" else codes.view(torch.float8_e4m3fn).float()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = np.random.default_rng(seed)
    s = {"case": c, "eps": 1e-6}
    if c["op"] == "tables":
        _prepare_tables(c, s, host, dev)
        return s
    if c["op"] == "verify":
        _prepare_verify(c, s, g, host, dev)
        return s
    t = TYPES[c["dtype"]]
    new, kv = _lengths(c)
    H, D, page = c["kv_heads"], c["dim"], c["page"]
    table, _, pages = _pool([-(-k // page) for k in kv], 3, host)
    s["table"] = torch.from_numpy(np.maximum(table, 0)).to(dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["max_q_len"] = max(new)
    s["cu_q"] = None
    if len(set(new)) > 1:
        s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
    # a cache as appends leave it: every page and head in a power of two that holds its largest element
    for x in "kv":
        held = torch.randn((pages, H, page, D), generator=g, device=dev)
        held *= 0.5 + torch.rand((pages, H, 1, 1), generator=g, device=dev)
        s[x + "_scale"] = _power_of_two(held.abs().amax((2, 3)) / LARGEST[c["kind"]])
        s[x + "_cache"] = _coded(held / s[x + "_scale"][:, :, None, None], c["kind"])
        del held
    if c["op"] == "attention":
        s["q"] = (torch.randn((sum(new), c["q_heads"], D), generator=g, device=dev) * 1.5).to(t)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    # a projection's output: keys and values of a token side by side; they grow with the channel as trained ones do
    kv_new = torch.randn((sum(new), 2 * H, D), generator=g, device=dev)
    kv_new *= 0.25 + 1.5 * torch.rand((2 * H, D), generator=g, device=dev)
    kv_new = kv_new.to(t)
    s["k"], s["v"] = kv_new[:, :H], kv_new[:, H:]
    s["positions"] = torch.cat([torch.arange(k - n, k, dtype=torch.int32) for n, k in zip(new, kv)]).to(dev)
    R = c["rotary"]
    base = 1e4 if seed % 2 else 1e6
    s["inv_freq"] = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R) if R else None
    s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(t) if c["norm"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_tables(s):
    page, width, n_tok = s["case"]["page"], s["table"].shape[1], s["n_tok"]
    dev = s["table"].device
    length, new, held = s["lengths"].long(), s["new"].long(), s["held"].long()
    B = length.numel()
    end = new.cumsum(0)
    need = (length + new + page - 1) // page
    fits = ((end <= n_tok) | (new == 0)) & (need <= width)
    surplus = torch.where(fits, (held - need).clamp(min=0), 0)
    take = torch.where(fits, (need - held).clamp(min=0), 0)
    left, back = s["n_free"].long(), surplus.sum()
    served = fits & ((take == 0) | (take.cumsum(0) <= left + back))
    take = torch.where(served, take, 0)
    # pages that come back, in order, and then the free ones from the top of the stack
    seq = torch.arange(B, device=dev)
    back_of, take_of = seq.repeat_interleave(surplus), seq.repeat_interleave(take)
    at = torch.arange(back_of.numel(), device=dev) - (surplus.cumsum(0) - surplus)[back_of]
    returned = s["table"][back_of, need[back_of] + at]
    k = torch.arange(take_of.numel(), device=dev)
    n_back, n_take = back_of.numel(), take_of.numel()
    stack = s["free"]
    from_stack = stack[(left - 1 - (k - n_back)).clamp(min=0, max=stack.numel() - 1)]
    pages = torch.where(k < n_back, returned[k.clamp(max=n_back - 1)], from_stack) if n_back else from_stack
    place = held[take_of] + k - (take.cumsum(0) - take)[take_of]
    s["table"][take_of, place] = pages
    r = torch.arange(n_take, max(n_back, n_take), device=dev)
    stack[left + r - n_take] = returned[r]
    s["n_free"].copy_(left + n_back - n_take)
    s["held"].copy_(torch.where(served, need, held))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), end]).clamp(max=n_tok)
    kv_len = torch.where(served, length + new, 0)
    tok = torch.arange(n_tok, device=dev)
    b = torch.searchsorted(cu[1:], tok, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    there &= served[b]
    pos = torch.where(there, length[b] + tok - cu[b], 0)
    slots = torch.where(there, s["table"][b, (pos // page).clamp(max=width - 1)].long() * page + pos % page, -1)
    return slots, pos.int(), cu.int(), kv_len.int(), (~served).sum().int()[None]


def _rotated(x, weight, s):
    """RMS norm (where there is a weight) and rotation of [T, H, D] in 32 bits; angles in 64."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    R = c["rotary"]
    if not R:
        return x
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    head, rest = x[..., :R], x[..., R:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., :R // 2], head[..., R // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([head, rest], -1)


def _token_places(s):
    """Request and key of every new token."""
    T, B = s["k"].shape[0], s["kv_len"].numel()
    tok = torch.arange(T, device=s["k"].device)
    start = torch.arange(B + 1, device=tok.device) * s["max_q_len"] if s["cu_q"] is None else s["cu_q"].long()
    b = torch.searchsorted(start[1:], tok, right=True)
    return b, s["kv_len"].long()[b] - start[1:][b] + tok


def _plain_append_one(x, codes, scale, page, place, kind):
    """Rows x [T, H, D] to their places, with the pages' scales grown where they have to be."""
    pages, H = scale.shape
    most = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    # rows held before
    first = torch.full((pages,), codes.shape[2], device=x.device).scatter_reduce(0, page, place, "amin")
    need = _power_of_two(most / LARGEST[kind])
    grown = torch.where((first > 0)[:, None], torch.maximum(scale, need), need)
    named = torch.zeros(pages, dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    held, head = (named[:, None] & (first > 0)[:, None] & (grown > scale)).nonzero(as_tuple=True)
    row = torch.arange(codes.shape[2], device=x.device)
    ratio = (scale[held, head] / grown[held, head])[:, None, None]
    old = codes[held, head]
    codes[held, head] = torch.where((row < first[held][:, None])[..., None], _coded(_value(old, kind) * ratio, kind), old)
    scale.copy_(torch.where(named[:, None], grown, scale))
    by = torch.where(scale[page] > 0, scale[page], 1.0)[..., None]
    codes[page, :, place] = _coded(x / by, kind)


def _plain_append(s):
    c = s["case"]
    b, key = _token_places(s)
    page, place = s["table"].long()[b, key // c["page"]], key % c["page"]
    _plain_append_one(_rotated(s["k"], s["k_weight"], s), s["k_cache"], s["k_scale"], page, place, c["kind"])
    _plain_append_one(s["v"].float(), s["v_cache"], s["v_scale"], page, place, c["kind"])


def _plain_attention(s):
    c = s["case"]
    table, page, H, D = s["table"].long(), c["page"], c["kv_heads"], c["dim"]
    B, L = table.shape[0], table.shape[1] * page
    G = c["q_heads"] // H

    def cached(x):
        r = _value(s[x + "_cache"][table], c["kind"]) * s[x + "_scale"][table][..., None, None]
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


def _plain_verify(s):
    c, dev = s["case"], s["target"].device
    p, q, N, B = s["target"], s["draft_probs"], s["draft"].numel(), c["seqs"]
    if s["cu_draft"] is None:
        cu = torch.arange(B + 1, device=dev) * (N // B)
    else:
        cu = s["cu_draft"].long()
    t, d = torch.arange(N, device=dev), s["draft"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    chance = s["uniform"].double() * (1.0 if q is None else q[t, d].double())
    refused = chance >= p[t + b, d].double()
    # drafts of each request before its first refused one
    count = cu.diff()
    kept = count.scatter_reduce(0, b[refused], (t - cu[b])[refused], "amin")
    row, at = cu[:-1] + kept + torch.arange(B, device=dev), (cu[:-1] + kept).clamp(max=max(N - 1, 0))
    w = p[row].double()
    more = kept < count
    if N:
        if q is None:
            less = w.scatter(1, d[at][:, None], 0.0)
        else:
            less = (w - q[at].double()).clamp(min=0.0)
        use = more & (less.sum(-1) > 0)  # a refused draft's token may be the only one
        w = torch.where(use[:, None], less, w)
    upto = w.cumsum(-1)
    last = (upto <= s["last_uniform"].double()[:, None] * upto[:, -1:]).sum(-1)
    tokens = torch.full((N + B,), -1, dtype=torch.int32, device=dev)
    ok = (t - cu[b]) < kept[b]
    tokens[t + b] = torch.where(ok, s["draft"], -1)
    tokens[row] = last.int()
    return tokens, kept.int()


def run(s):
    c = s["case"]
    if own:
        import hashed_gram_memory_amd as hg

        if c["op"] == "tables":
            out = hg.page_tables(s["lengths"], s["new"], s["table"], s["held"], s["free"], s["n_free"], c["page"], s["n_tok"])
        elif c["op"] == "verify":
            return hg.verify_draft(s["target"], s["draft"], s["uniform"], s["last_uniform"], draft_probs=s["draft_probs"],
                                   cu_draft=s["cu_draft"])
        elif c["op"] == "append":
            hg.kv_append_pages(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                               s["kv_len"], cu_q=s["cu_q"], max_q_len=s["max_q_len"], positions=s["positions"],
                               inv_freq=s["inv_freq"], k_weight=s["k_weight"], eps=s["eps"], interleaved=c["interleaved"])
        else:
            return hg.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], cu_q=s["cu_q"],
                                      max_q_len=s["max_q_len"], scale=s["scale"], window=c["window"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=c["lse"])
    elif c["op"] == "tables":
        out = _plain_tables(s)
    elif c["op"] == "verify":
        return _plain_verify(s)
    elif c["op"] == "append":
        _plain_append(s)
    else:
        return _plain_attention(s)
    if c["op"] == "tables":
        slots, positions, cu_q, kv_len, n_short = out
        return {"slots": slots, "positions": positions, "cu_q": cu_q, "kv_len": kv_len, "n_short": n_short,
                "table": s["table"], "held": s["held"], "free": s["free"], "n_free": s["n_free"]}
    of = (lambda x: x) if c["kind"] == "int8" else (lambda x: x.view(torch.float8_e4m3fn))  # noqa: E731
    return {"k": of(s["k_cache"]), "v": of(s["v_cache"]), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_tables(c, s):
    page, width, n_tok = c["page"], s["table"].shape[1], s["n_tok"]
    length, new, held = (s[x].tolist() for x in ("lengths", "new", "held"))
    table, stack, n_free = s["table"].cpu().numpy().copy(), s["free"].tolist(), int(s["n_free"])
    need = [-(-(a + n) // page) for a, n in zip(length, new)]
    slots, positions, cu, kv_len, short = [-1] * n_tok, [0] * n_tok, [0], [], 0
    fits, tokens = [], 0
    for b, n in enumerate(new):
        tokens += n
        fits.append((tokens <= n_tok or n == 0) and need[b] <= width)
        cu.append(min(tokens, n_tok))
    back = []
    for b, h in enumerate(held):
        if fits[b] and h > need[b]:
            back += table[b, need[b]:h].tolist()
            held[b] = need[b]
    pool = back + stack[:n_free][::-1]
    dealt = wanted = 0
    for b, n in enumerate(new):
        ok = fits[b]
        if ok and need[b] > held[b]:
            wanted += need[b] - held[b]
            ok = wanted <= len(pool)
            if ok:
                table[b, held[b]:need[b]] = pool[dealt:wanted]
                dealt, held[b] = wanted, need[b]
        short += not ok
        kv_len.append(length[b] + n if ok else 0)
        if ok:
            for i in range(n):
                p = length[b] + i
                slots[cu[b] + i], positions[cu[b] + i] = int(table[b, p // page]) * page + p % page, p
    over = back[dealt:]
    left = n_free - max(dealt - len(back), 0)
    stack[left:left + len(over)] = over
    left += len(over)
    dev, i32 = s["table"].device, torch.int32
    to = lambda x, t=i32: torch.tensor(x, dtype=t, device=dev)  # noqa: E731
    return {"slots": to(slots, torch.int64), "positions": to(positions), "cu_q": to(cu), "kv_len": to(kv_len),
            "n_short": to([short]), "table": to(table), "held": to(held), "free": to(stack), "n_free": to([left])}


def _exact_verify(c, s):
    k = _drafts(c)
    tokens, kept = [], []
    at = 0
    draft, u, last = s["draft"].tolist(), s["uniform"].tolist(), s["last_uniform"].tolist()
    for b, n in enumerate(k):
        row = at + b
        took, w = 0, None
        for i in range(n):
            p, d = s["target"][row + i].double(), draft[at + i]
            if s["draft_probs"] is None:
                q = torch.zeros_like(p)
                q[d] = 1.0
            else:
                q = s["draft_probs"][at + i].double()
            if u[at + i] * float(q[d]) < float(p[d]):
                took += 1
                continue
            w = torch.relu(p - q)
            w = w if float(w.sum()) > 0 else p
            break
        if w is None:
            w = s["target"][row + n].double()
        total = torch.cumsum(w, 0)
        j = int(torch.searchsorted(total, last[b] * total[-1], right=True))
        tokens += draft[at:at + took] + [j] + [-1] * (n - took)
        kept.append(took)
        at += n
    dev = s["target"].device
    return torch.tensor(tokens, dtype=torch.int32, device=dev), torch.tensor(kept, dtype=torch.int32, device=dev)


def _turned(x, weight, s):
    """The norm and the rotation of [T, H, D], each pair as a complex number."""
    c, x = s["case"], x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * weight.double()
    R = c["rotary"]
    if R == 0:
        return x
    pair = x[..., :R].unflatten(-1, (R // 2, 2) if c["interleaved"] else (2, R // 2))
    if not c["interleaved"]:
        pair = pair.transpose(-1, -2)
    turn = torch.exp(1j * (s["positions"].double().unsqueeze(-1) * s["inv_freq"]))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn.unsqueeze(1))
    if not c["interleaved"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., R:]), dim=-1)


def _nearest(x, kind):
    """The value nearest to x that a code stands for, ties to even."""
    if kind == "int8":
        return torch.round(x)
    # 3 bits below the leading one, steps of 2^-9 at least
    grid = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / grid) * grid


def _exact_append(c, s):
    new, kv = _lengths(c)
    page, kind, found = c["page"], c["kind"], {}
    table = s["table"].cpu()
    for name, x in (("k", _turned(s["k"], s["k_weight"], s)), ("v", s["v"].double())):
        raw = s[name + "_cache"]
        held = (raw if kind == "int8" else raw.view(torch.float8_e4m3fn)).double()
        scale = s[name + "_scale"].double()
        at = 0
        for b, (n, length) in enumerate(zip(new, kv)):
            a = length - n
            while a < length:  # page by page
                e = min(length, (a // page + 1) * page)
                rows = x[at:at + e - a].transpose(0, 1)  # [H, n, D]
                p, r = int(table[b, a // page]), a % page
                least = rows.abs().amax((1, 2)) / LARGEST[kind]
                step = torch.where(least > 0, torch.exp2(torch.ceil(torch.log2(least.clamp(min=1e-300)))), 0.0)
                step = torch.where(step / 2 >= least, step / 2, step)  # where the logarithm was rounded up
                if r:
                    step = torch.maximum(step, scale[p])
                    held[p, :, :r] = torch.where((step > scale[p])[:, None, None],
                                                 _nearest(held[p, :, :r] * (scale[p] / step)[:, None, None], kind),
                                                 held[p, :, :r])
                held[p, :, r:r + e - a] = _nearest(rows / torch.where(step > 0, step, 1.0)[:, None, None], kind)
                scale[p] = step
                at += e - a
                a = e
        found[name] = held.to(torch.int8) if kind == "int8" else held
        found[name + "_scale"] = scale
    return {x: found[x] for x in ("k", "v", "k_scale", "v_scale")}


def _exact_attention(c, s):
    new, kv = _lengths(c)
    page, H, G = c["page"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    outs, lses = [], []
    at = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        if n == 0:
            continue
        low = max(0, length - n + 1 - c["window"]) if c["window"] else 0
        key = torch.arange(low, length, device=s["q"].device)
        ids = s["table"][b].long()[key // page]
        newest = torch.arange(length - n, length, device=key.device)
        seen = key <= newest[:, None]
        if c["window"]:
            seen &= newest[:, None] - key < c["window"]
        heads, logs = [], []
        for h in range(H):
            kk, vv = (_value(s[x + "_cache"][ids, h, key % page], c["kind"]).double()
                      * s[x + "_scale"][ids, h].double()[:, None] for x in "kv")
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


def exact(c, seed):
    s = prepare(c, seed)
    return {"tables": _exact_tables, "append": _exact_append, "attention": _exact_attention,
            "verify": _exact_verify}[c["op"]](c, s)
