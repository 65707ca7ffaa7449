"""The calls of a drafting step at the edges of their use: refusals of the binding, streams, workspaces, gradients, places past
2^32 elements, and slots with the other append."""
import math

import pytest
import torch
import torch.autograd.forward_ad as fwd

import drafts_oracle as do
import serving_oracle as so
from gpu_support import lib
from test_gpu_serving import BF16, F16, P_SPLIT, _close
from test_gpu_append_pages import _batch, _call, _device
from test_gpu_verify_draft import _batch as _drafts

pytestmark = pytest.mark.gpu

I32, F32 = torch.int32, torch.float32


def _z(*s, t=I32):
    return torch.zeros(s, dtype=t, device="cuda")


def _good():
    """Arguments that each call takes."""
    return {
        "kv_append_pages": dict(k=_z(2, 2, 64, t=BF16), v=_z(2, 2, 64, t=BF16), k_cache=_z(4, 2, 16, 64, t=torch.int8),
                                v_cache=_z(4, 2, 16, 64, t=torch.int8), k_scale=_z(4, 2, t=F32), v_scale=_z(4, 2, t=F32),
                                block_table=_z(2, 3), kv_len=_z(2) + 5, cu_q=torch.arange(3, dtype=I32, device="cuda"),
                                positions=_z(2), inv_freq=_z(16, t=torch.float64), k_weight=_z(64, t=BF16)),
        "page_tables": dict(lengths=_z(2), new_tokens=_z(2) + 1, block_table=_z(2, 3), held=_z(2),
                            free_pages=torch.arange(9, dtype=I32, device="cuda"), n_free=_z(1) + 9, page_size=16, n_tok=2),
        "verify_draft": dict(target=_z(5, 40, t=F32) + 0.1, draft=_z(3), uniform=_z(3, t=F32), last_uniform=_z(2, t=F32),
                             draft_probs=_z(3, 40, t=F32) + 0.1, cu_draft=torch.tensor([0, 1, 3], dtype=I32, device="cuda")),
    }


BAD = {
    "kv_append_pages": [
        dict(k=_z(2, 2, 64)), dict(k=_z(2, 2, 64, t=F16)), dict(k=_z(2, 3, 64, t=BF16)), dict(v=_z(3, 2, 64, t=BF16)),
        dict(v_cache=_z(4, 2, 16, 64, t=torch.uint8)), dict(k_cache=_z(4, 2, 16, 32, t=torch.int8)),
        dict(k_cache=_z(4, 16, 2, 64, t=torch.int8).transpose(1, 2)), dict(k_scale=_z(4, 2, 16, t=F32)), dict(v_scale=_z(4, 3, t=F32)),
        dict(v_scale=_z(4, 2, t=torch.float64)), dict(k_scale=_z(2, 4, t=F32).T), dict(block_table=_z(2, 3, t=torch.int64)),
        dict(block_table=_z(3, 2).T), dict(kv_len=_z(3)), dict(kv_len=_z(2, t=torch.int64)), dict(cu_q=_z(2)), dict(positions=None),
        dict(positions=_z(3)), dict(inv_freq=_z(16, t=F32)), dict(inv_freq=_z(3, t=torch.float64)), dict(k_weight=_z(32, t=BF16)),
        dict(eps=-1.0), dict(max_q_len=-2), dict(cu_q=None, block_table=_z(3, 3), kv_len=_z(3)),
        dict(k_cache=_z(4, 2, 16, 64, t=BF16), v_cache=_z(4, 2, 16, 64, t=BF16)),
        dict(k_cache=_z(4, 2, 16, 64, t=torch.uint8), v_cache=_z(4, 2, 16, 64, t=torch.uint8), k_scale=_z(4, 2, 16, t=F32),
             v_scale=_z(4, 2, 16, t=F32)),
    ],
    "page_tables": [
        dict(lengths=_z(3)), dict(lengths=_z(2, t=torch.int64)), dict(new_tokens=_z(1)), dict(block_table=_z(3, 2).T),
        dict(block_table=_z(2, 3, t=torch.int64)), dict(block_table=_z(1, 3).expand(2, 3)), dict(held=_z(2, 1)),
        dict(free_pages=_z(3, 3)), dict(free_pages=_z(18)[::2]), dict(n_free=_z(2)), dict(n_free=_z(1, t=torch.int64)),
        dict(page_size=0), dict(page_size=-16), dict(page_size=24), dict(page_size=2 ** 40 + 16), dict(n_tok=-1), dict(n_tok=2 ** 31),
        dict(new_tokens=None, n_tok=3), dict(workspace=_z(4, t=F32)), dict(lengths=None),
    ],
    "verify_draft": [
        dict(target=_z(5, 40)), dict(target=_z(5, 40, t=torch.float64)), dict(target=_z(40, 5, t=F32).T), dict(target=_z(2, 40, t=F32)),
        dict(target=_z(5, 0, t=F32), draft_probs=_z(3, 0, t=F32)), dict(draft=_z(3, t=torch.int64)), dict(draft=_z(3, 1)),
        dict(uniform=_z(2, t=F32)), dict(uniform=_z(3, t=torch.float64)), dict(last_uniform=_z(3, t=F32)),
        dict(draft_probs=_z(3, 41, t=F32)), dict(draft_probs=_z(5, 40, t=F32)), dict(draft_probs=_z(3, 40, t=BF16)),
        dict(cu_draft=_z(2)), dict(cu_draft=None), dict(uniform=None), dict(target=torch.zeros((5, 40))),
    ],
} if torch.cuda.is_available() else {}


@pytest.mark.parametrize("name", ["kv_append_pages", "page_tables", "verify_draft"])
def test_binding_refuses(name):
    hg = lib()
    call, good = getattr(hg, name), _good()[name]
    call(**good)
    before = {k: v.clone() for k, v in good.items() if torch.is_tensor(v)}
    for i, bad in enumerate(BAD[name]):
        with pytest.raises((ValueError, TypeError, hg.EngramError)):
            call(**dict(good, **bad))
            pytest.fail(f"call {i} was accepted")
    torch.cuda.synchronize()
    assert all(torch.equal(good[k], v) for k, v in before.items())
    with pytest.raises(ValueError, match="kv_append_pages"):
        g = _good()["kv_append_pages"]
        hg.kv_append(g["k"], g["v"], g["k_cache"], g["v_cache"], _z(2, t=torch.int64), k_scale=g["k_scale"], v_scale=g["v_scale"])


@pytest.mark.parametrize("name", ["kv_append_pages", "verify_draft"])
def test_tensors_with_a_derivative(name):
    hg = lib()
    call, args = getattr(hg, name), _good()[name]
    for k in [k for k, x in args.items() if x.is_floating_point()]:
        with pytest.raises(ValueError, match="gradient"):
            call(**dict(args, **{k: args[k].clone().requires_grad_()}))
        with torch.no_grad():
            call(**dict(args, **{k: args[k].clone().requires_grad_()}))
        with fwd.dual_level(), pytest.raises(ValueError, match="gradient"):
            call(**dict(args, **{k: fwd.make_dual(args[k], torch.ones_like(args[k]))}))
    outs = call(**args)
    assert outs is None or not any(x.requires_grad for x in outs)


def test_streams():
    """Behind work of the stream that is given, by object and by handle, with nothing waited for between."""
    hg = lib()
    s = _drafts([3, 1], 50000, F32, 3)
    d = {k: v.cuda() for k, v in s.items()}
    want = hg.verify_draft(d["target"], d["draft"], d["uniform"], d["last"], d["q"], d["cu"])
    b = _batch(6, "int8", BF16, 64, 2, 8, [11], [13])
    e, f = _device(b), _device(b)
    _call(e)
    t = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    big = torch.ones(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream, 0):
        on = torch.cuda.default_stream() if given == 0 else side
        late = {k: torch.zeros_like(v) for k, v in d.items()}
        kv, lens, state = torch.zeros_like(f["kv"]), t(0, 0), (_z(2, 9), t(0, 0), torch.arange(30, dtype=I32, device="cuda"), t(30))
        cache = [f[x].clone() for x in ("k_cache", "v_cache", "k_scale", "v_scale")]
        torch.cuda.synchronize()
        with torch.cuda.stream(on):
            for _ in range(6):
                big.mul_(1.0)
            for k in d:
                late[k].copy_(d[k])
            kv.copy_(f["kv"])
            lens.copy_(t(20, 3))
        got = hg.verify_draft(late["target"], late["draft"], late["uniform"], late["last"], late["q"], late["cu"], stream=given)
        hg.kv_append_pages(kv[:, :2], kv[:, 2:], *cache, f["table"], f["kv_len"], f["cu"], stream=given)
        tables = hg.page_tables(lens, None, *state, 8, 2, stream=given)
        on.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, e[y]) for x, y in zip(cache, ("k_cache", "v_cache", "k_scale", "v_scale")))
        assert tables[3].tolist() == [21, 4] and tables[1].tolist() == [20, 3]
        torch.cuda.synchronize()


def test_workspaces_that_are_given():
    """Of the size that is asked for, with any contents; one byte less is refused; two calls on two streams have their own."""
    hg = lib()
    s = _drafts([3, 1], 70001, BF16, 3)
    d = {k: v.cuda() for k, v in s.items()}
    args = (d["target"], d["draft"], d["uniform"], d["last"], d["q"], d["cu"])
    need = hg.verify_draft_workspace(*args)
    want = hg.verify_draft(*args)
    t = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    state = lambda: (t([50] * 2000), None, _z(2000, 9), t([6] * 2000), torch.arange(5000, dtype=I32, device="cuda"), t([5000]), 8, 8000)  # noqa: E731
    more = hg.page_tables_workspace(*state())
    assert need > 0 and more > 0
    want_tables = hg.page_tables(*state())
    for fill in (0, 255):
        ws, ws2 = (torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in (need, more))
        assert all(torch.equal(x, y) for x, y in zip(hg.verify_draft(*args, workspace=ws), want))
        assert all(torch.equal(x, y) for x, y in zip(hg.page_tables(*state(), workspace=ws2), want_tables))
        for bad in (ws[:-1], ws[1:]):
            with pytest.raises(hg.EngramError):
                hg.verify_draft(*args, workspace=bad)
        with pytest.raises(hg.EngramError):
            hg.page_tables(*state(), workspace=ws2[:-1])
    two = [torch.cuda.Stream() for _ in range(2)]
    other = {k: v.cuda() for k, v in _drafts([3, 1], 70001, BF16, 4).items()}
    args2 = (other["target"], other["draft"], other["uniform"], other["last"], other["q"], other["cu"])
    want2 = hg.verify_draft(*args2)
    torch.cuda.synchronize()
    for _ in range(10):
        got, got2 = hg.verify_draft(*args, stream=two[0]), hg.verify_draft(*args2, stream=two[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + got2, want + want2))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 6, 60])
def test_pages_past_4_gigabytes(kind, new):
    """Appends and attention on pages past 2^32 codes, K and V in one pool, against a small cache with the same rows."""
    hg = lib()
    D, H, page = 256, 1, 1024
    far = 17000  # pages of 2 * 256 KiB apart: 8.9 GB
    s = _batch(new, kind, BF16, D, H, page, [new, 1], [1500, 30], 128, True)
    d = _device(s)
    _call(d, max_q_len=new)
    q = torch.randn((new + 1, 4, D), generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    want = hg.paged_attention(q, d["k_cache"], d["v_cache"], d["table"], d["kv_len"], d["cu"], new, k_scale=d["k_scale"],
                              v_scale=d["v_scale"], return_lse=True)
    pool = torch.empty((far, 2, H, page, D), dtype=d["k_cache"].dtype, device="cuda")
    e = dict(_device(s), k_scale=_z(far, H, t=F32), v_scale=_z(far, H, t=F32))
    shift = torch.tensor([far - 1 - 3 * i for i in range(s["k_cache"].shape[0])])
    for x, side in (("k", 0), ("v", 1)):
        pool[shift.cuda(), side] = s[x + "_cache"].cuda()
        e[x + "_cache"] = pool[:, side]
        e[x + "_scale"][shift.cuda()] = s[x + "_scale"].cuda()
    e["table"] = torch.where(s["table"] < 2 ** 29, shift[s["table"].clamp(max=shift.numel() - 1).long()].int(), s["table"]).cuda()
    _call(e, max_q_len=new)
    for x in "kv":
        assert torch.equal(e[x + "_cache"][shift.cuda()], d[x + "_cache"]) and torch.equal(e[x + "_scale"][shift.cuda()], d[x + "_scale"])
    got = hg.paged_attention(q, e["k_cache"], e["v_cache"], e["table"], e["kv_len"], e["cu"], new, k_scale=e["k_scale"],
                             v_scale=e["v_scale"], return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_rows_past_2_to_the_32():
    """Probabilities whose rows lie past 2^32 elements; a table whose rows do."""
    hg = lib()
    s = _drafts([2, 3], 5000, BF16, 8)
    want = do.verify(s["target"], s["draft"], s["uniform"], s["last"], s["q"], s["cu"])
    stride = 2 ** 30
    base = torch.empty(6 * stride + 5000, dtype=BF16, device="cuda")
    far = base.as_strided((7, 5000), (stride, 1))
    far.copy_(s["target"])
    got = hg.verify_draft(far, s["draft"].cuda(), s["uniform"].cuda(), s["last"].cuda(), s["q"].cuda(), s["cu"].cuda())
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
    q = base.as_strided((5, 5000), (stride, 1))
    q.copy_(s["q"])
    got = hg.verify_draft(s["target"].cuda(), s["draft"].cuda(), s["uniform"].cuda(), s["last"].cuda(), q, s["cu"].cuda())
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
    del far, q
    table = base.view(torch.int32).as_strided((6, 4), (2 ** 29, 1))
    table[:] = -3
    t = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    for n_tok in (30, 9000):
        table[:] = -3
        table[3, 0], table[5, :3] = 40, t(50, 51, 52)
        out = hg.page_tables(t(0, 0, 0, 8, 0, 0), t(0, 3, 0, 9, 0, 9), table, t(0, 0, 0, 1, 0, 3), t(7, 8, 9), t(3), 8, n_tok)
        assert out[0][:21].tolist() == [416, 417, 418, *range(72, 80), 64, *range(400, 408), 408][:21]
        assert table.tolist() == [[-3] * 4, [52, -3, -3, -3], [-3] * 4, [40, 9, 8, -3], [-3] * 4, [50, 51, 52, -3]]


def test_slots_with_the_append_by_slots():
    """Slots and positions into a 16-bit cache by kv_append, and the attention of the same call's lengths."""
    hg = lib()
    H, D, page, lens = 2, 64, 8, [37, 1, 20]
    g = torch.Generator().manual_seed(4)
    t = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    table, held, free, n_free, lengths = _z(3, 6) - 1, t(0, 0, 0), torch.arange(12, dtype=I32, device="cuda"), t(12), t(0, 0, 0)
    kc, vc = (torch.full((12, H, page, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    rows = [[], [], []]
    for new in ([30, 0, 20], [6, 1, 0], [1, 0, 0]):
        n_tok = sum(new) + 5
        kv = torch.randn((n_tok, 2 * H, D), generator=g).to(BF16)
        slots, positions, cu, kv_len, short = hg.page_tables(lengths, t(*new), table, held, free, n_free, page, n_tok)
        assert int(short) == 0
        hg.kv_append(kv[:, :H].cuda(), kv[:, H:].cuda(), kc, vc, slots)
        lengths = kv_len
        at = 0
        for b, n in enumerate(new):
            assert positions[at:at + n].tolist() == list(range(len(rows[b]), len(rows[b]) + n))
            rows[b] += list(kv[at:at + n])
            at += n
    assert lengths.tolist() == lens
    q = torch.randn((3, 4, D), generator=g).to(BF16)
    out, lse = hg.paged_attention(q.cuda(), kc, vc, table, lengths, return_lse=True)
    for b, n in enumerate(lens):
        kv = torch.stack(rows[b])
        pages = torch.nn.functional.pad(kv, (0, 0, 0, 0, 0, -n % page)).unflatten(0, (-1, page)).transpose(1, 2)
        o, l, mass, move = so.attention(q[b:b + 1], pages[:, :H], pages[:, H:], torch.arange(pages.shape[0])[None], torch.tensor([n]),
                                        torch.tensor([0, 1]), D ** -0.5, 0)
        bound, _ = so.attention_bounds(o, l, mass, move, BF16, P_SPLIT[BF16])
        _close(out[b:b + 1], o, bound, b)


def test_a_stack_of_the_most_pages():
    """2^30 free pages, and five requests that want 2^28 - 512 each: four get them, the fifth is not taken for served because
    the sum of what they want is past what a call may have."""
    hg = lib()
    page, each = 8, (2 ** 31 - 4096) // 8
    table = torch.full((5, each), -3, dtype=I32, device="cuda")
    free = torch.arange(1 << 30, dtype=I32, device="cuda")
    n_free = torch.tensor([1 << 30], dtype=I32, device="cuda")
    lengths, held = torch.full((5,), each * page, dtype=I32, device="cuda"), _z(5)
    out = hg.page_tables(lengths, _z(5), table, held, free, n_free, page, 1 << 21)
    assert out[3].tolist() == [each * page] * 4 + [0] and out[4].tolist() == [1] and held.tolist() == [each] * 4 + [0]
    assert n_free.tolist() == [(1 << 30) - 4 * each]
    for b in range(4):  # from the top of the stack down
        want = torch.arange((1 << 30) - 1 - b * each, (1 << 30) - 1 - (b + 1) * each, -1, dtype=I32, device="cuda")
        assert torch.equal(table[b], want)
    assert (table[4] == -3).all()
