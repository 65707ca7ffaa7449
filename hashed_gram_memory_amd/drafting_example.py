"""Decoding with drafted tokens next to the lookup, all of it on the GPU: ``python -m hashed_gram_memory_amd.drafting_example``.

A batch of requests goes on from step to step without the host: a step drafts
a few tokens of each request, makes its pages fit (page_tables), looks the
tokens up (lookup), appends their keys and values to a cache of 8-bit codes
with one scale for each page and head (kv_append_pages), attends
(paged_attention), and keeps the drafts that the target's probabilities bear
out, with one token more (verify_draft).  The lengths that the next step
begins with are those that came out, so a captured step is replayed while the
requests grow, are short of pages and wait, and give pages of refused drafts
back.  Weights and tables are random; the drafter knows the last token only.
"""
from __future__ import annotations

import argparse
import time

import torch

import hashed_gram_memory_amd as hg
import hashed_gram_memory_amd.serving  # noqa: F401  (loaded here and not by the first call, which is timed)
from hashed_gram_memory_amd.attention_example import random_plan


class Pool:
    """The pages of up to ``n_seq`` requests, as page_tables keeps them: tables, pages held, and a stack of free ones."""

    def __init__(self, n_seq: int, n_pages: int, page_size: int, max_len: int):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page_size = page_size
        self.lengths = torch.zeros(n_seq, **i32)
        self.held = torch.zeros(n_seq, **i32)
        self.block_table = torch.full((n_seq, -(-max_len // page_size)), -1, **i32)
        self.free_pages = torch.arange(n_pages, **i32)
        self.n_free = torch.full((1,), n_pages, **i32)

    def place(self, new: torch.Tensor | None, n_tok: int):
        """Pages for ``new`` tokens of each request (None: equally many); positions, cu_q and kv_len of the step."""
        _, positions, cu_q, kv_len, _ = hg.page_tables(self.lengths, new, self.block_table, self.held, self.free_pages,
                                                       self.n_free, self.page_size, n_tok)
        return positions, cu_q, kv_len


class Layer:
    """q, k, v from what the lookup reads, attention over codes, and a head that stands for the rest of a model."""

    def __init__(self, plan: hg.Plan, pool: Pool, vocab: int, n_q_heads: int = 32, n_kv_heads: int = 8, head_dim: int = 128,
                 int8: bool = True, window: int = 0, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.plan, self.pool, self.window, self.vocab = plan, pool, window, vocab
        self.heads, self.kv_heads, self.dim = n_q_heads, n_kv_heads, head_dim
        width = hg.N_MODULES * hg.ROW_BYTES
        normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.w_qkv = (normal(width, (n_q_heads + 2 * n_kv_heads) * head_dim) / width ** 0.5).bfloat16().cuda()
        self.w_head = (normal(n_q_heads * head_dim, vocab) * 6 / (n_q_heads * head_dim) ** 0.5).bfloat16().cuda()
        self.q_weight, self.k_weight = ((1 + 0.1 * normal(head_dim)).bfloat16().cuda() for _ in range(2))
        self.inv_freq = (1e4 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).cuda()
        n_pages = pool.free_pages.numel()
        shape = (n_pages, n_kv_heads, pool.page_size, head_dim)
        self.cache = [torch.zeros(shape, dtype=torch.int8 if int8 else torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(shape[:2], device="cuda") for _ in range(2)]

    def project(self, ids: torch.Tensor, history: torch.Tensor | None = None):
        """q, k, v [n_tok, heads, head_dim] of ids [n_seq, seq_len]: slices of one product, with its strides."""
        memory = hg.lookup(self.plan, ids, history).flatten(1)
        memory = memory * torch.rsqrt(memory.square().mean(-1, keepdim=True) + 1e-6)
        qkv = (memory.bfloat16() @ self.w_qkv).unflatten(-1, (-1, self.dim))
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def attend(self, q, k, v, positions, cu_q, kv_len, max_q_len: int) -> torch.Tensor:
        """The layer's output [n_tok, n_q_heads, head_dim]; k and v are in the cache afterwards."""
        q, _ = hg.qk_norm_rope(q, None, positions, self.inv_freq, q_weight=self.q_weight)
        hg.kv_append_pages(k, v, *self.cache, *self.scales, self.pool.block_table, kv_len, cu_q, max_q_len, positions,
                           self.inv_freq, self.k_weight)
        return hg.paged_attention(q, *self.cache, self.pool.block_table, kv_len, cu_q, max_q_len, window=self.window,
                                  k_scale=self.scales[0], v_scale=self.scales[1])

    def probabilities(self, out: torch.Tensor) -> torch.Tensor:
        return torch.softmax((out.flatten(1) @ self.w_head).float(), -1)


class Drafting:
    """One step of all requests, ``drafts`` drafted tokens each, with everything on the device so that it can be captured.
    The random numbers of a step are filled in before it (draw)."""

    def __init__(self, layer: Layer, ids: torch.Tensor, history: torch.Tensor, drafts: int, seed: int = 0):
        n = ids.shape[0]
        g = torch.Generator().manual_seed(seed)
        self.layer, self.drafts = layer, drafts
        self.ids, self.history = ids.clone(), history.clone()       # the token that comes next, those before it
        self.drafter = (torch.randn((layer.vocab, layer.vocab), generator=g) * 2).cuda()
        self.choose = torch.zeros((drafts, n), device="cuda")       # for the drafts,
        self.uniform = torch.zeros(n * drafts, device="cuda")       # whether they stay,
        self.last = torch.zeros(n, device="cuda")                   # and the token after them
        self.emitted = torch.zeros(n, dtype=torch.int64, device="cuda")

    def draw(self, generator: torch.Generator | None = None) -> None:
        for x in (self.choose, self.uniform, self.last):
            x.uniform_(generator=generator)

    def step(self) -> dict:
        layer, pool, n, k = self.layer, self.layer.pool, self.ids.shape[0], self.drafts
        tokens, probs = [self.ids], []
        for i in range(k):
            q = torch.softmax(self.drafter[tokens[-1][:, 0].long()], -1)
            upto = q.cumsum(-1)
            word = (upto <= self.choose[i][:, None] * upto[:, -1:]).sum(-1, keepdim=True).clamp(max=layer.vocab - 1)
            tokens.append(word.int())
            probs.append(q)
        fed = torch.cat(tokens, 1)
        draft, q = fed[:, 1:].reshape(-1), torch.stack(probs, 1).flatten(0, 1)

        positions, cu_q, kv_len = pool.place(None, n * (k + 1))
        qkv = layer.project(fed, self.history)
        out = layer.attend(*qkv, positions, cu_q, kv_len, k + 1)
        target = layer.probabilities(out)
        emitted, accepted = hg.verify_draft(target, draft, self.uniform, self.last, q)

        served = kv_len > 0  # the others wait for pages
        count = torch.where(served, accepted + 1, 0)
        after = torch.cat([self.history, fed], 1).long()  # the tokens before the next one end at place 3 + accepted
        at = torch.where(served, accepted + 1, 0).long()[:, None]
        self.history.copy_(after.gather(1, at + torch.arange(3, device=at.device)))
        following = emitted.view(n, k + 1).gather(1, accepted[:, None].long())
        self.ids.copy_(torch.where(served[:, None], following, self.ids))
        pool.lengths += count
        self.emitted += count
        return {"fed": fed, "draft": draft, "q": q, "out": out, "target": target, "tokens": emitted, "accepted": accepted,
                "kv_len": kv_len, "positions": positions}


def prompts_in(layer: Layer, prompts: list[torch.Tensor]):
    """Prompts into the cache in one call, but for the last token of each: (that token, the three before it).  Refused where
    the pool or a table does not hold them all; the requests' lengths are then as they were."""
    new = [p.numel() - 1 for p in prompts]
    q, k, v = (torch.cat(x) for x in zip(*(layer.project(p[None]) for p in prompts)))
    keep = torch.cat([torch.arange(p.numel(), device="cuda") < p.numel() - 1 for p in prompts])
    counts = torch.tensor(new, dtype=torch.int32, device="cuda")
    positions, cu_q, kv_len = layer.pool.place(counts, sum(new))
    short = (kv_len != counts).nonzero()[:, 0].tolist()
    if short:  # without its prompt a request would go on from its last token alone
        raise RuntimeError(f"no room for the prompts of the requests {short}: more pages or a wider table are needed")
    if sum(new):
        layer.attend(q[keep], k[keep], v[keep], positions, cu_q, kv_len, max(new))
    layer.pool.lengths.copy_(kv_len)
    last = torch.stack([p[-1:] for p in prompts])
    return last, torch.stack([torch.nn.functional.pad(p[:-1], (3, 0))[-3:] for p in prompts])


def captured(drafting: Drafting):
    """A graph of one step, and what it gives.  One step is taken eagerly: what a graph holds has to have run before."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        drafting.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = drafting.step()
    return graph, out


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1024, help="tokens of the longest prompt")
    ap.add_argument("--drafts", type=int, default=5, help="drafted tokens of a step")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--e4m3", action="store_true", help="hold the cache in FP8 E4M3 (default: int8)")
    args = ap.parse_args(argv)
    n = args.requests
    most = args.prompt + (args.steps + 1) * (args.drafts + 1)
    pool = Pool(n, n * -(-most // args.page), args.page, most)
    layer = Layer(random_plan(), pool, args.vocab, int8=not args.e4m3)
    g = torch.Generator().manual_seed(1)
    lens = [max(2, args.prompt * (b + 1) // n) for b in range(n)]
    prompts = [torch.randint(0, args.vocab, (m,), generator=g, dtype=torch.int32).cuda() for m in lens]
    drafting = Drafting(layer, *prompts_in(layer, prompts), args.drafts)
    drafting.draw()
    graph, _ = captured(drafting)
    torch.cuda.synchronize()
    before, start = drafting.emitted.clone(), time.perf_counter()
    for _ in range(args.steps):
        drafting.draw()
        graph.replay()
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start
    came = int((drafting.emitted - before).sum())
    print(f"prompts: {sum(lens)} tokens of {n} requests")
    print(f"drafting: {args.steps} steps of {args.drafts} drafts, {seconds * 1e6 / args.steps:.1f} us a step, "
          f"{came / (args.steps * n):.2f} tokens a step and request; {int(pool.n_free)} pages free")


if __name__ == "__main__":
    main()
