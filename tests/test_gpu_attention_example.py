"""The attention layer next to the lookup: prompts in chunks, then tokens from a graph."""
import pytest
import torch

import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, _close

pytestmark = pytest.mark.gpu


def _layer(e4m3, n_seq, page, most, heads, kv_heads, dim, window=0):
    lib()
    from hashed_gram_memory_amd import attention_example as ex
    n_pages = n_seq * -(-most // page) + 1
    requests = ex.Requests(n_seq, n_pages, page, most)
    return ex, ex.AttentionLayer(ex.random_plan(256), requests, n_pages, heads, kv_heads, dim, e4m3, window)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_in_pieces(e4m3):
    """Chunks, short runs, single tokens and requests without a token in one call, against the whole in 64 bits."""
    hg = lib()
    lens, page = [150, 1, 37], 16
    ex, layer = _layer(e4m3, len(lens), page, 160, 6, 2, 64)
    g = torch.Generator().manual_seed(5)
    ids = [torch.randint(0, 5000, (1, n), generator=g, dtype=torch.int32).cuda() for n in lens]
    qkv = [layer.project(i) for i in ids]
    got = [[] for _ in lens]
    at = [0] * len(lens)
    for new in ([100, 1, 0], [1, 0, 30], [49, 0, 1], [0, 0, 6]):
        batch = layer.requests.step(new)
        parts = [torch.cat([x[i][a:a + m] for x, a, m in zip(qkv, at, new)]) for i in range(3)]
        out = layer.attend(*parts, batch)
        for b, piece in enumerate(out.split(new)):
            got[b].append(piece)
        at = [a + m for a, m in zip(at, new)]
    assert layer.requests.lens == lens

    host = lambda x: None if x is None else x.cpu()  # noqa: E731
    table, cache, scales = layer.requests.host, layer.cache.cpu(), [host(s) for s in layer.scales]
    freq, eps = layer.inv_freq.cpu(), 1e-6
    for b, n in enumerate(lens):
        pos = torch.arange(n, dtype=torch.int32)
        q, k, v = (x.cpu() for x in qkv[b])
        # the cache holds the request's keys and values where its pages say
        rows, fp = so.norm_rope(k, layer.k_weight.cpu(), eps, pos, freq, False)
        where = table[b].long()[pos // page], pos.long() % page
        for side, want, fp in ((0, rows, fp), (1, v.double(), torch.zeros_like(fp))):
            held = cache[side][where[0], :, where[1]]
            if e4m3:
                scale = scales[side][where[0], :, where[1]].double()[..., None]
                amax = want.abs().amax(-1, keepdim=True)
                held = held.view(torch.float8_e4m3fn).double() * scale
                # half a step of a code (steps of 2^-9 below 2^-6), and what fp32 moved the row and its scale by
                moved = fp + fp.amax(-1, keepdim=True) + 16 * so.U32 * amax
                bound = want.abs() * 2.0 ** -4 + amax / 448 * 2.0 ** -10 + 2 * moved
            else:
                bound = so.rounding_bound(want, fp, BF16)
            _close(held, want, bound, ("cache", b, side))
        # the output, from the queries as they are turned and the cache as it stands
        turned, _ = hg.qk_norm_rope(qkv[b][0], None, pos.cuda(), layer.inv_freq, q_weight=layer.q_weight)
        out, lse, mass, move = so.attention(turned.cpu(), cache[0], cache[1], table[b:b + 1], torch.tensor([n]),
                                            torch.tensor([0, n]), 64 ** -0.5, 0, *scales)
        bound, _ = so.attention_bounds(out, lse, mass, move, BF16, so.half_step(BF16))
        _close(torch.cat(got[b]), out, bound, ("out", b))


def test_tokens_from_a_graph():
    """Replays of a captured step against eager steps from the same state, with other work between."""
    n, most = 3, 64
    ex, layer = _layer(False, n, 8, most, 4, 2, 128, window=20)
    g = torch.Generator().manual_seed(9)
    lens = [19, 1, 30]
    ids = [torch.randint(0, 5000, (1, m), generator=g, dtype=torch.int32).cuda() for m in lens]
    parts = [torch.cat(x) for x in zip(*(layer.project(i) for i in ids))]
    layer.attend(*parts, layer.requests.step(lens))
    layer.requests.reserve(most)
    first = torch.stack([i[0, -1:] for i in ids])
    history = torch.stack([torch.nn.functional.pad(i[0, :-1], (3, 0))[-3:] for i in ids])
    eager = ex.Decoder(layer, first, history, 5000)
    want = [(eager.step().clone(), eager.ids.clone()) for _ in range(6)]
    captured = ex.Decoder(layer, first, history, 5000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.step()
    for k in range(6):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k][0]) and torch.equal(captured.ids, want[k][1]), k
        layer.project(ids[2])
        torch.cuda.synchronize()
    assert captured.kv_len.tolist() == [m + 6 for m in lens]


def test_the_command(capsys):
    lib()
    from hashed_gram_memory_amd import attention_example as ex
    ex.main(["--requests", "3", "--prompt", "40", "--chunk", "16", "--tokens", "4", "--e4m3"])
    said = capsys.readouterr().out
    assert "prompts: 79 tokens of 3 requests in 3 calls" in said and "decode: 3 requests" in said
