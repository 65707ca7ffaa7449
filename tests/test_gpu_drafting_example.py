"""The drafting step together, next to the lookup: prompts in, then steps, eager and from a graph."""
import pytest
import torch

import drafts_oracle as do
import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, P_SPLIT, _close

pytestmark = pytest.mark.gpu


def _start(int8, lens, drafts, pages, page=8, vocab=64, heads=4, kv_heads=2, dim=64, window=0):
    lib()
    from hashed_gram_memory_amd import drafting_example as ex
    pool = ex.Pool(len(lens), pages, page, 160)
    layer = ex.Layer(ex.random_plan(256), pool, vocab, heads, kv_heads, dim, int8, window)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, vocab, (n,), generator=g, dtype=torch.int32).cuda() for n in lens]
    return ex, pool, layer, ex.Drafting(layer, *ex.prompts_in(layer, prompts), drafts), prompts


def _held_once(pool):
    held = pool.held.tolist()
    mine = [p for row, h in zip(pool.block_table.tolist(), held) for p in row[:h]]
    free = pool.free_pages.tolist()[:int(pool.n_free)]
    assert sorted(mine + free) == list(range(pool.free_pages.numel()))


def _check_step(ex, pool, layer, drafting, before, out, int8):
    """What a step gave, from the state `before` it: verification against the form, the output against the cache as it is."""
    n, k = drafting.ids.shape[0], drafting.drafts
    host = {x: y.cpu() for x, y in out.items()}
    cu = torch.arange(n + 1) * k
    tokens, accepted = do.verify(host["target"], host["draft"], drafting.uniform.cpu(), drafting.last.cpu(), host["q"], cu)
    assert host["tokens"].tolist() == tokens and host["accepted"].tolist() == accepted
    served = host["kv_len"] > 0
    want = before["lengths"] + torch.where(served, torch.tensor(accepted) + 1, 0)
    assert pool.lengths.cpu().tolist() == want.tolist()
    assert host["kv_len"][served].tolist() == (before["lengths"] + k + 1)[served].tolist()
    for b in range(n):
        told = [int(x) for x in host["fed"][b, :accepted[b] + 1]] + [tokens[b * (k + 1) + accepted[b]]] if served[b] else [int(before["ids"][b])]
        seq = (before["history"][b].tolist() + told)
        assert drafting.ids[b].tolist() == seq[-1:] and drafting.history[b].tolist() == seq[-4:-1]
    # the attention over the cache as it stands, for the requests that were served
    turned, _ = lib().qk_norm_rope(layer.project(out["fed"], before["history"].cuda())[0], None, out["positions"], layer.inv_freq,
                                   q_weight=layer.q_weight)
    kind = "int8" if int8 else "e4m3"
    kc, vc = (do.values(c.cpu(), kind) * s.cpu().double()[:, :, None, None] for c, s in zip(layer.cache, layer.scales))
    o, lse, mass, move = so.attention(turned.cpu(), kc, vc, pool.block_table.cpu(), host["kv_len"], torch.arange(n + 1) * (k + 1),
                                      layer.dim ** -0.5, layer.window)
    bound, _ = so.attention_bounds(o, lse, mass, move, BF16, P_SPLIT[BF16])
    _close(out["out"], o, bound, "out")


@pytest.mark.parametrize("int8,window", [(True, 0), (False, 20)])
def test_steps(int8, window):
    lens = [40, 2, 17, 9]
    ex, pool, layer, drafting, prompts = _start(int8, lens, 4, 80, window=window)
    assert pool.lengths.tolist() == [n - 1 for n in lens]
    _held_once(pool)
    g = torch.Generator(device="cuda").manual_seed(7)
    some = set()
    for _ in range(6):
        drafting.draw(g)
        before = {"lengths": pool.lengths.cpu(), "ids": drafting.ids.cpu(), "history": drafting.history.cpu()}
        out = drafting.step()
        _check_step(ex, pool, layer, drafting, before, out, int8)
        _held_once(pool)
        some.update(out["accepted"].tolist())
    assert len(some) > 1


def test_the_cache_holds_what_was_kept():
    """After several steps the cache's rows are the keys and values of the tokens that stayed, within their codes."""
    lens = [30, 5]
    ex, pool, layer, drafting, prompts = _start(True, lens, 3, 60)
    g = torch.Generator(device="cuda").manual_seed(1)
    kept = [p[:-1].tolist() for p in prompts]
    for _ in range(5):
        drafting.draw(g)
        out = drafting.step()
        for b in range(2):
            kept[b] += out["fed"][b, :int(out["accepted"][b]) + 1].tolist()
    assert pool.lengths.tolist() == [len(x) for x in kept]
    for b, ids in enumerate(kept):
        _, k, v = layer.project(torch.tensor([ids], dtype=torch.int32, device="cuda"))
        pos = torch.arange(len(ids), dtype=torch.int32)
        rows, fp = so.norm_rope(k.cpu(), layer.k_weight.cpu(), 1e-6, pos, layer.inv_freq.cpu(), False)
        page, place = pool.block_table[b].cpu().long()[pos // 8], pos.long() % 8
        for side, (want, off) in enumerate(((rows, fp), (v.cpu().double(), torch.zeros_like(rows)))):
            scale = layer.scales[side].cpu().double()[page][..., None]
            got = layer.cache[side].cpu().double()[page, :, place] * scale
            # an int8 code is off by less than a step of its page however often the page grew
            _close(got, want, scale + off, (b, side))


@pytest.mark.parametrize("pages", [80, 9])
def test_steps_from_a_graph(pages):
    """Replays against eager steps of a twin, with other work between; with 9 pages requests wait for pages that never come."""
    lens = [30, 3, 20]
    ex, pool, layer, drafting, _ = _start(True, lens, 4, pages)
    _, pool2, layer2, twin, _ = _start(True, lens, 4, pages)
    for d in (drafting, twin):
        d.draw(torch.Generator(device="cuda").manual_seed(5))
    graph, out = ex.captured(drafting)
    twin.step()
    g = torch.Generator(device="cuda").manual_seed(6)
    waited = False
    for k in range(7):
        drafting.draw(g)
        for x, y in ((twin.choose, drafting.choose), (twin.uniform, drafting.uniform), (twin.last, drafting.last)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = twin.step()
        torch.cuda.synchronize()
        assert all(torch.equal(out[x], want[x]) for x in out), k
        for a, b in ((pool, pool2), (drafting, twin)):
            for x, y in vars(a).items():
                if torch.is_tensor(y):
                    assert torch.equal(y, vars(b)[x]), (k, x)
        assert all(torch.equal(a, b) for a, b in zip(layer.cache + layer.scales, layer2.cache + layer2.scales))
        waited |= bool((out["kv_len"] == 0).any())
        _held_once(pool)
    assert waited == (pages == 9)


def test_the_command(capsys):
    lib()
    from hashed_gram_memory_amd import drafting_example as ex
    ex.main(["--requests", "3", "--prompt", "40", "--drafts", "3", "--steps", "4", "--vocab", "512", "--e4m3"])
    said = capsys.readouterr().out
    assert "prompts: 79 tokens of 3 requests" in said and "drafting: 4 steps of 3 drafts" in said
