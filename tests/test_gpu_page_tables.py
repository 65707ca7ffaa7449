"""Page tables and slots from request lengths, against the plain form, entry by entry."""
import random

import pytest
import torch

import drafts_oracle as do
from gpu_support import lib

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _state(lengths, new, held, page, width, spare, room=None, seed=0):
    """A pool in random order: `held[b]` pages of each request, `spare` on the stack; marks in every other place."""
    rng = random.Random(seed)
    have = [min(max(h, 0), width) for h in held]
    order = list(range(sum(have) + spare))
    rng.shuffle(order)
    table, at = [], 0
    for h in have:
        table.append(order[at:at + h] + [-7] * (width - h))
        at += h
    stack = order[at:] + [-9] * ((len(order) if room is None else room) - spare)
    return {"lengths": lengths, "new": new, "table": table, "held": held, "stack": stack, "n_free": spare, "page": page}


def _call(s, n_tok, wide=0, uniform=False, **more):
    """The call on device copies: (outputs by name, the device state)."""
    t = lambda x: torch.tensor(x, dtype=I32).cuda()  # noqa: E731
    n, width = len(s["lengths"]), len(s["table"][0]) if s["table"] else 0
    base = torch.full((n, width + wide), -5, dtype=I32, device="cuda")  # rows further apart than they are wide
    base[:, :width] = torch.tensor(s["table"], dtype=I32).reshape(n, width).cuda()
    d = {"table": base[:, :width], "held": t(s["held"]), "free": t(s["stack"]), "n_free": t([s["n_free"]]), "base": base}
    got = lib().page_tables(t(s["lengths"]), None if uniform else t(s["new"]), d["table"], d["held"], d["free"], d["n_free"],
                            s["page"], n_tok, **more)
    out = dict(zip(("slots", "positions", "cu_q", "kv_len", "n_short"), got))
    out.update({k: d[k] for k in ("table", "held", "free", "n_free")})
    if wide:
        assert (base[:, width:] == -5).all()
    return out, d


def _check(s, n_tok, **more):
    want = do.page_tables(s["lengths"], s["new"], s["table"], s["held"], s["stack"], s["n_free"], s["page"], n_tok)
    got, d = _call(s, n_tok, **more)
    for k, x in want.items():
        assert got[k].cpu().tolist() == x, k
    assert got["slots"].dtype == torch.int64 and all(got[k].dtype == I32 for k in ("positions", "cu_q", "kv_len", "n_short"))
    return want, got, d


def _random(rng, n, most_len, most_new, page, scarce=1.0, surplus=0.2, room=None):
    lengths = [rng.choice([0, rng.randint(0, most_len)]) for _ in range(n)]
    new = [rng.choice([0, 1, rng.randint(0, most_new)]) for _ in range(n)]
    held = [-(-a // page) + (rng.randint(1, 3) if rng.random() < surplus else 0) for a in lengths]
    width = max([-(-(a + m) // page) for a, m in zip(lengths, new)] + held + [1])
    wanted = sum(max(-(-(a + m) // page) - h, 0) for a, m, h in zip(lengths, new, held))
    return _state(lengths, new, held, page, width, int(wanted * scarce) + (3 if scarce == 1.0 else 0), room, rng.random())


# requests, longest, new tokens, page, pages free (share of those wanted), share of requests with pages to give back
CASES = [(1, 0, 1, 16, 1.0, 0.0), (1, 100, 40, 8, 1.0, 1.0), (7, 50, 6, 16, 1.0, 0.3), (64, 500, 6, 16, 1.0, 0.1),
         (64, 500, 6, 16, 0.4, 0.0), (63, 300, 20, 8, 0.0, 0.5), (65, 90, 300, 32, 0.7, 0.9), (1024, 60, 8, 8, 0.8, 0.2),
         (1025, 60, 8, 8, 0.8, 0.2), (1000, 700, 40, 1024, 1.0, 0.2), (3000, 30, 9, 8, 0.5, 0.5), (5000, 20, 3, 8, 0.9, 0.3),
         (3, 4000, 9000, 16, 1.0, 0.5)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_tables(case):
    n, most_len, most_new, page, scarce, surplus = case
    rng = random.Random(n * 7 + page)
    for k in range(2):
        s = _random(rng, n, most_len, most_new, page, scarce, surplus)
        total = sum(s["new"])
        _check(s, total + k * 37, wide=3 * k)


def test_both_forms_agree():
    """The same requests just below and above the tokens that one workgroup takes: padding does not change a result."""
    s = _random(random.Random(5), 900, 200, 8, 8, 0.9, 0.3)
    assert sum(s["new"]) <= 8192
    a, b = _call(s, 8192)[0], _call(s, 8193)[0]
    for k in a:
        x, y = a[k], b[k]
        assert torch.equal(x, y[:8192] if k in ("slots", "positions") else y), k
    assert b["slots"][8192] == -1 and b["positions"][8192] == 0


@pytest.mark.parametrize("form", [0, 9000])
def test_who_is_served(form):
    """Requests that do not fit keep what they hold: too wide for the table, past the batch, without pages."""
    # the last one gives two pages back, so that three are there: the first takes two, the second would take four, the third
    # takes none, and the fourth, who would take one, comes after the second
    s = _state([0, 16, 5, 0, 40], [16, 17, 0, 8, 0], [0, 1, 1, 0, 7], 8, 7, 1)
    want, got, _ = _check(s, 41 + form)
    assert want["n_short"] == [2] and want["kv_len"] == [16, 0, 5, 0, 40]
    s = _state([0, 8, 3], [9, 1, 1], [0, 1, 1], 8, 1, 5)  # the first two need two pages, the table has one
    want, _, _ = _check(s, 11 + form)
    assert want["kv_len"] == [0, 0, 4] and want["n_short"] == [2]
    s = _state([3, 3, 3, 3], [2, 3, 1, 0], [1, 1, 1, 1], 8, 2, 5)  # the batch ends inside the second request's tokens
    if not form:
        want, _, _ = _check(s, 4)
        assert want["kv_len"] == [5, 0, 0, 3] and want["cu_q"] == [0, 2, 4, 4, 4]
    # lengths and counts below 0, pages held past the table, a stack that says more than it has
    s = _state([-5, 3, 7], [2, -4, 1], [-2, 9, 1], 8, 4, 2)
    s["n_free"] = 100
    s["stack"] = s["stack"][:2]
    _check(s, 8 + form)
    # pages that come back past the stack's room are dropped
    s = _state([0, 0], [0, 0], [4, 3], 8, 4, 1, room=3)
    want, _, _ = _check(s, form)
    assert want["n_free"] == [3]


@pytest.mark.parametrize("n_tok", [0, 5, 9000])
def test_no_request(n_tok):
    z = lambda *shape: torch.zeros(shape, dtype=I32, device="cuda")  # noqa: E731
    n_free = z(1) + 4
    slots, positions, cu, kv, short = lib().page_tables(z(0), z(0), z(0, 3), z(0), z(6), n_free, 16, n_tok)
    assert (slots == -1).all() and (positions == 0).all() and slots.numel() == n_tok
    assert cu.tolist() == [0] and kv.numel() == 0 and short.tolist() == [0] and n_free.tolist() == [4]


def test_equal_requests_without_counts():
    s = _state([5, 16, 0], [4, 4, 4], [1, 1, 0], 8, 3, 6)
    a, b = _call(s, 12)[0], _call(s, 12, uniform=True)[0]
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_lengths_at_their_limits():
    """Keys up to 2^31 - 4096 of a request, and sums of tokens past 2^32."""
    page = 1024
    most = 2 ** 31 - 4096
    width = most // page
    table = torch.zeros((3, width), dtype=I32, device="cuda")
    table[:, -1] = torch.tensor([7, 2 ** 31 - 1, 9], dtype=I32, device="cuda")
    t = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    held, n_free = t(width, width, width), t(0)
    out = lib().page_tables(t(most - 1, most - 1, most), t(1, 1, 1), table, held, t(1, 2), n_free, page, 4)
    assert out[0].tolist() == [7 * page + 1023, (2 ** 31 - 1) * page + 1023, -1, -1]
    assert out[3].tolist() == [most, most, 0] and out[4].tolist() == [1]
    big = 2 ** 31 - 1
    s = _state([0] * 5, [3, big, big, big, 0], [0] * 5, 8, 4, 9)
    want, got, _ = _check(s, 10)
    assert want["kv_len"] == [3, 0, 0, 0, 0] and want["cu_q"] == [0, 3, 10, 10, 10, 10]


def test_a_pool_through_many_steps():
    """Requests that come, grow, lose refused tokens and end: every page is held once or free, and the slots are theirs."""
    rng = random.Random(3)
    n, page, width, pages = 40, 8, 12, 150
    t = lambda x: torch.tensor(x, dtype=I32).cuda()  # noqa: E731
    lengths = [0] * n
    table, held, free, n_free = torch.full((n, width), -1, dtype=I32, device="cuda"), t([0] * n), t(range(pages)), t([pages])
    host = {"table": table.tolist(), "held": [0] * n, "stack": list(range(pages)), "n_free": pages}
    for _ in range(25):
        new = [rng.choice([0, 1, 6, 30]) if a + 30 <= width * page else 0 for a in lengths]
        want = do.page_tables(lengths, new, host["table"], host["held"], host["stack"], host["n_free"], page, 600)
        got = lib().page_tables(t(lengths), t(new), table, held, free, n_free, page, 600)
        for k, x in zip(("slots", "positions", "cu_q", "kv_len", "n_short"), got):
            assert x.tolist() == want[k], k
        assert table.tolist() == want["table"] and held.tolist() == want["held"] and n_free.tolist() == want["n_free"]
        host = {"table": want["table"], "held": want["held"], "stack": want["free"], "n_free": want["n_free"][0]}
        mine = [p for r, h in zip(host["table"], host["held"]) for p in r[:h]] + host["stack"][:host["n_free"]]
        assert sorted(mine) == list(range(pages))
        for b in range(n):
            if want["kv_len"][b]:
                kept = rng.randint(0, new[b]) if new[b] else 0
                lengths[b] = lengths[b] + kept if rng.random() > 0.15 else 0


def test_replays():
    """A captured call, replayed over changed lengths with other work between, against eager calls on copies."""
    hg = lib()
    rng = random.Random(8)
    for n_tok in (64, 9000):
        s = _random(rng, 30, 80, 20, 8, 1.0, 0.2)
        t = lambda x: torch.tensor(x, dtype=I32).cuda()  # noqa: E731
        args = [t(s["lengths"]), t([0] * 30), t(s["table"]), t(s["held"]), t(s["stack"]), t([s["n_free"]])]
        hg.page_tables(*[x.clone() for x in args], 8, n_tok)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = hg.page_tables(*args, 8, n_tok)
        for k in range(4):
            args[1].copy_(t([rng.randint(0, 3) for _ in range(30)]))
            copies = [x.clone() for x in args]
            want = hg.page_tables(*copies, 8, n_tok)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, want)), (n_tok, k)
            assert all(torch.equal(x, y) for x, y in zip(args, copies)), (n_tok, k)
            args[0].copy_(out[3])
            torch.cuda.synchronize()
