"""An attention layer next to the lookup, as a server would drive it: ``python -m hashed_gram_memory_amd.attention_example``.

Prompts are read in chunks of mixed lengths, then all requests decode together,
one token a step, from a HIP graph.  Each step looks the new tokens up
(lookup), projects what the lookup read to q, k and v, appends the keys and
values to a paged cache (kv_append), turns the queries (qk_norm_rope) and
attends over the cache (paged_attention).  Weights and tables are random.
"""
from __future__ import annotations

import argparse
import time
from dataclasses import dataclass

import torch

import hashed_gram_memory_amd as hg
import hashed_gram_memory_amd.serving  # noqa: F401  (loaded here and not by the first call, which is timed)


@dataclass
class Batch:
    """The new tokens of one call: where they are, and what each request's keys are after them."""
    positions: torch.Tensor        # int32 [n_tok]
    slots: torch.Tensor            # int64 [n_tok]
    kv_len: torch.Tensor           # int32 [n_seq]
    cu_q: torch.Tensor | None      # int32 [n_seq + 1]; None: one token each
    max_q_len: int


class Requests:
    """Lengths and pages of up to ``n_seq`` requests; pages are dealt as requests grow."""

    def __init__(self, n_seq: int, n_pages: int, page_size: int, max_len: int, device="cuda"):
        self.page_size, self.device = page_size, device
        self.lens = [0] * n_seq
        self.free = list(range(n_pages))[::-1]
        self.pages: list[list[int]] = [[] for _ in range(n_seq)]
        # an entry that is no page is never read
        self.host = torch.full((n_seq, -(-max_len // page_size)), -1, dtype=torch.int32)
        self.block_table = self.host.to(device)

    def reserve(self, length: int) -> None:
        """Pages for all requests up to ``length`` tokens, so that a graph can append to them."""
        self._grow([length] * len(self.lens))

    def _grow(self, lens: list[int]) -> None:
        for b, n in enumerate(lens):
            while len(self.pages[b]) * self.page_size < n:
                page = self.free.pop()
                self.host[b, len(self.pages[b])] = page
                self.pages[b].append(page)
        self.block_table.copy_(self.host)

    def step(self, new: list[int]) -> Batch:
        """``new[b]`` more tokens of request b."""
        after = [n + m for n, m in zip(self.lens, new)]
        self._grow(after)
        pos = [torch.arange(n, e) for n, e in zip(self.lens, after)]
        slots = torch.cat([self.host[b, p // self.page_size].long() * self.page_size + p % self.page_size
                           for b, p in enumerate(pos)])
        cu = torch.tensor([0] + new).cumsum(0)
        self.lens = after
        to = lambda x, t: x.to(t).to(self.device)  # noqa: E731
        return Batch(to(torch.cat(pos), torch.int32), to(slots, torch.int64), to(torch.tensor(after), torch.int32),
                     to(cu, torch.int32), max(new))


class AttentionLayer:
    """q, k, v from what the lookup reads; norm, rotation, cache and attention by the serving operators."""

    def __init__(self, plan: hg.Plan, requests: Requests, n_pages: int, n_q_heads: int = 32, n_kv_heads: int = 8,
                 head_dim: int = 128, e4m3: bool = False, window: int = 0, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.plan, self.requests, self.window = plan, requests, window
        self.heads, self.kv_heads, self.dim = n_q_heads, n_kv_heads, head_dim
        width = hg.N_MODULES * hg.ROW_BYTES
        self.w_qkv = (torch.randn((width, (n_q_heads + 2 * n_kv_heads) * head_dim), generator=g) / width ** 0.5).bfloat16().cuda()
        self.q_weight = (1 + 0.1 * torch.randn(head_dim, generator=g)).bfloat16().cuda()
        self.k_weight = (1 + 0.1 * torch.randn(head_dim, generator=g)).bfloat16().cuda()
        self.inv_freq = (1e4 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).cuda()
        pool = (2, n_pages, n_kv_heads, requests.page_size)
        self.cache = torch.zeros((*pool, head_dim), dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        self.scales = torch.zeros(pool, device="cuda") if e4m3 else (None, None)

    def project(self, ids: torch.Tensor, history: torch.Tensor | None = None):
        """q, k, v [n_tok, heads, head_dim] of ids [n_seq, seq_len]: slices of one product, with its strides."""
        memory = hg.lookup(self.plan, ids, history).flatten(1)
        memory = memory * torch.rsqrt(memory.square().mean(-1, keepdim=True) + 1e-6)
        qkv = (memory.bfloat16() @ self.w_qkv).unflatten(-1, (-1, self.dim))
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def attend(self, q, k, v, batch: Batch, workspace: torch.Tensor | None = None) -> torch.Tensor:
        """The layer's output [n_tok, n_q_heads, head_dim]; k and v are in the cache afterwards."""
        q, _ = hg.qk_norm_rope(q, None, batch.positions, self.inv_freq, q_weight=self.q_weight)
        hg.kv_append(k, v, *self.cache, batch.slots, batch.positions, self.inv_freq, self.k_weight,
                     k_scale=self.scales[0], v_scale=self.scales[1])
        return hg.paged_attention(q, *self.cache, self.requests.block_table, batch.kv_len, batch.cu_q, batch.max_q_len,
                                  window=self.window, k_scale=self.scales[0], v_scale=self.scales[1], workspace=workspace)


class Decoder:
    """One token of every request, with everything on the device: ids, positions, slots and lengths move on by themselves,
    so that a captured step can be replayed.  Bits of the output stand in for a model's head and sampling."""

    def __init__(self, layer: AttentionLayer, ids: torch.Tensor, history: torch.Tensor, vocab: int):
        r = layer.requests
        self.layer, self.ids, self.history, self.vocab = layer, ids.clone(), history.clone(), vocab
        self.positions = torch.tensor(r.lens, dtype=torch.int32, device="cuda")
        self.kv_len = self.positions.clone()
        q = torch.empty((len(r.lens), layer.heads, layer.dim), dtype=torch.bfloat16, device="cuda")
        bytes_ = hg.paged_attention_workspace(q, *layer.cache, r.block_table, self.kv_len, window=layer.window,
                                              k_scale=layer.scales[0], v_scale=layer.scales[1])
        self.workspace = torch.empty(max(bytes_, 1), dtype=torch.uint8, device="cuda")

    def step(self) -> torch.Tensor:
        r, at = self.layer.requests, self.positions.long()
        page = r.block_table.gather(1, (at // r.page_size)[:, None])[:, 0].long()
        self.kv_len.copy_(self.positions + 1)
        batch = Batch(self.positions, page * r.page_size + at % r.page_size, self.kv_len, None, 1)
        q, k, v = self.layer.project(self.ids, self.history)
        out = self.layer.attend(q, k, v, batch, self.workspace)
        chosen = out[:, 0, :1].view(torch.int16).int() & 0x7FFF
        self.history.copy_(torch.cat([self.history[:, 1:], self.ids], 1))
        self.ids.copy_(chosen % self.vocab)
        self.positions += 1
        return out


def random_plan(rows: int = 1 << 14, seed: int = 0) -> hg.Plan:
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 0x70, (hg.N_SUB, rows, hg.ROW_BYTES), dtype=torch.uint8, device="cuda", generator=g)
    sign = torch.randint(0, 2, codes.shape, dtype=torch.uint8, device="cuda", generator=g) << 7
    return hg.Plan(codes | sign, torch.rand((hg.N_SUB, rows), device="cuda", generator=g) + 0.5)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2048, help="tokens of the longest prompt")
    ap.add_argument("--chunk", type=int, default=512, help="new tokens of a request in one call")
    ap.add_argument("--tokens", type=int, default=64, help="tokens to decode")
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--e4m3", action="store_true", help="hold the cache in FP8 E4M3")
    args = ap.parse_args(argv)
    n, vocab = args.requests, 8192
    most = args.prompt + args.tokens
    n_pages = n * -(-most // args.page)
    requests = Requests(n, n_pages, args.page, most)
    layer = AttentionLayer(random_plan(), requests, n_pages, e4m3=args.e4m3)
    g = torch.Generator().manual_seed(1)
    left = [max(1, args.prompt * (b + 1) // n) for b in range(n)]
    prompts = [torch.randint(0, vocab, (m,), generator=g, dtype=torch.int32).cuda() for m in left]
    qkv = [layer.project(p[None]) for p in prompts]  # one lookup a prompt

    torch.cuda.synchronize()
    start, calls = time.perf_counter(), 0
    while any(left):
        new = [min(m, args.chunk) for m in left]
        at = requests.lens[:]
        batch = requests.step(new)
        parts = [torch.cat([x[i][a:a + m] for x, a, m in zip(qkv, at, new)]) for i in range(3)]
        layer.attend(*parts, batch)
        left = [m - d for m, d in zip(left, new)]
        calls += 1
    torch.cuda.synchronize()
    total = sum(requests.lens)
    print(f"prompts: {total} tokens of {n} requests in {calls} calls, {(time.perf_counter() - start) * 1e3:.2f} ms")

    requests.reserve(most)
    last = torch.stack([p[-1:] for p in prompts])
    history = torch.stack([torch.nn.functional.pad(p[:-1], (3, 0))[-3:] for p in prompts])
    decoder = Decoder(layer, last, history, vocab)
    # what a graph holds has to have run before; this step is the first token's
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decoder.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decoder.step()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.tokens - 1):
        graph.replay()
    torch.cuda.synchronize()
    steps = max(args.tokens - 1, 1)
    print(f"decode: {n} requests, {(time.perf_counter() - start) * 1e6 / steps:.1f} us a step; "
          f"next ids {decoder.ids[:8, 0].tolist()}")


if __name__ == "__main__":
    main()
