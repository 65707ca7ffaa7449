"""Verification of drafts against the plain form in 64 bits: the same words."""
import math

import pytest
import torch

import drafts_oracle as do
from gpu_support import lib

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _batch(counts, vocab, dtype, seed, sharp=3.0, certain=False, far=0.6):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(counts), len(counts)
    logits = sharp * torch.randn((n + b, vocab), generator=g)
    seq = torch.tensor([i for i, c in enumerate(counts) for _ in range(c)], dtype=torch.long)
    s = {"target": torch.softmax(logits, -1).to(dtype), "uniform": torch.rand(n, generator=g), "last": torch.rand(b, generator=g)}
    q = torch.softmax(logits[torch.arange(n) + seq] + far * torch.randn((n, vocab), generator=g), -1)
    s["q"] = None if certain else q.to(dtype)
    s["draft"] = (torch.multinomial(q, 1, generator=g)[:, 0] if n else torch.zeros(0)).int()
    if certain and n:
        s["draft"] = q.argmax(-1).int()
    s["cu"] = torch.tensor([0] + counts).cumsum(0).int()
    return s


def _run(s, by_offsets=True, **more):
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    return lib().verify_draft(c(s["target"]), c(s["draft"]), c(s["uniform"]), c(s["last"]), draft_probs=c(s["q"]),
                              cu_draft=c(s["cu"]) if by_offsets else None, **more)


def _check(s, **more):
    tokens, accepted = do.verify(s["target"], s["draft"], s["uniform"], s["last"], s["q"], s["cu"])
    got = _run(s, **more)
    assert got[1].tolist() == accepted
    assert got[0].tolist() == tokens
    assert got[0].dtype == got[1].dtype == torch.int32
    return tokens, accepted


CASES = [
    # drafts of each request, vocabulary, dtype, certain
    ([0], 1, F32, False), ([1], 1, BF16, False), ([1], 2, F32, True), ([5], 1000, F32, False),
    ([0, 3, 0, 7, 1], 333, BF16, False), ([2, 2, 2], 16, F16, False), ([4, 0], 17, F16, True),
    ([5] * 9, 16384, F32, False), ([5, 0, 2], 16385, BF16, False), ([3, 1], 32768, F16, False), ([3, 1], 32768, F32, True),
    ([3, 0, 6], 32769, F32, False), ([2, 5], 99091, BF16, False), ([1, 2], 129280, F32, False), ([2, 1], 262147, F16, True),
    ([70, 1, 200], 50, F32, False), ([1] * 300, 40, F32, False), ([2] * 70, 40000, BF16, True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_verify(case):
    counts, vocab, dtype, certain = case
    some = set()
    for k in range(3):
        s = _batch(counts, vocab, dtype, vocab + len(counts) + k, certain=certain)
        _, accepted = _check(s)
        some.update(accepted)
        if len(set(counts)) == 1:
            a, b = _run(s), _run(s, by_offsets=False)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        again = _run(s)
        assert torch.equal(again[0], _run(s)[0])
    assert len(counts) < 9 or len(some) > 1


@pytest.mark.parametrize("vocab", [9, 33000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_random_numbers_at_their_ends(vocab, dtype):
    """0 and the last number below 1, numbers outside, NaN: a word with a weight always comes out."""
    s = _batch([1, 1, 0, 2, 1, 0], vocab, dtype, 5)
    s["target"][:, :3] = 0.0  # words without a weight at both ends
    s["target"][:, -2:] = 0.0
    below = 1 - 2.0 ** -24
    for v in (0.0, below, 1.0, 7.0, -1.0, math.nan):
        s["last"][:] = v
        for u in (0.0, below):
            s["uniform"][:] = u
            tokens, _ = _check(s)
            assert all(x == -1 or x < vocab for x in tokens)
    # a draft that the target does not know is refused at u = 0 too, and one that it gives all to is kept
    s["target"][:] = 0.0
    s["target"][:, 4] = 1.0
    s["uniform"][:] = 0.0
    s["draft"][:] = 1
    assert set(_check(s)[1]) == {0}
    s["uniform"][:] = below
    s["draft"][:] = 4
    assert _check(s)[1] == [1, 1, 0, 2, 1, 0]


@pytest.mark.parametrize("vocab", [40, 40000])
@pytest.mark.parametrize("certain", [False, True])
def test_rows_that_leave_nothing(vocab, certain):
    """A refused draft whose residual is empty takes the target's row; a row of zeros, NaN or infinities has no word."""
    s = _batch([1, 1, 1, 0, 0, 1, 1], vocab, F32, 9, certain=certain)
    p, d = s["target"], s["draft"].long()
    p[0] = 0.0
    p[0, d[0]] = 0.5  # all that the target gives is the refused word
    if not certain:
        s["q"][0] = 0.0
        s["q"][0, d[0]] = 1.0
    p[2] = 0.0                  # a zero row
    p[4] = math.nan
    p[6, 3] = math.inf          # a request without drafts
    p[7] = 0.0
    p[8, : vocab // 2] = math.nan   # NaN weigh nothing
    p[9, : vocab // 2] = -1.0
    s["uniform"][:] = 0.9999
    tokens, accepted = _check(s)
    assert tokens[0] == int(d[0]) and accepted[:3] == [0, 0, 0]
    assert tokens[2] == -1 and tokens[4] == -1 and tokens[6] == -1 and tokens[7] == -1
    assert all(x >= vocab // 2 or x == -1 for x in tokens[8:10])


@pytest.mark.parametrize("vocab", [50, 70000])
def test_drafts_that_are_no_words(vocab):
    for certain in (False, True):
        s = _batch([3, 2, 1], vocab, F32, 3, certain=certain)
        s["uniform"][:] = 0.0
        s["draft"][1], s["draft"][3], s["draft"][5] = -1, vocab, 2 ** 31 - 1
        _, accepted = _check(s)
        assert accepted == [1, 0, 0]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides(dtype):
    """Rows further apart than they are wide, on odd places, and the same row for all."""
    s = _batch([2, 3], 4099, dtype, 21)
    want = _run(s)
    for pad, at in ((1, 1), (5, 3), (64, 0)):
        wide = {}
        for k in ("target", "q"):
            base = torch.full((s[k].shape[0], 4099 + pad), math.nan, dtype=dtype).cuda()
            base[:, at:at + 4099] = s[k].cuda()
            wide[k] = base[:, at:at + 4099]
        got = lib().verify_draft(wide["target"], s["draft"].cuda(), s["uniform"].cuda(), s["last"].cuda(), wide["q"], s["cu"].cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = s["target"][:1].cuda()
    many = dict(s, target=one.cpu().expand(7, 4099))
    got = lib().verify_draft(one.expand(7, 4099), s["draft"].cuda(), s["uniform"].cuda(), s["last"].cuda(), s["q"].cuda(), s["cu"].cuda())
    tokens, accepted = do.verify(many["target"], s["draft"], s["uniform"], s["last"], s["q"], s["cu"])
    assert got[0].tolist() == tokens and got[1].tolist() == accepted


@pytest.mark.parametrize("vocab", [7, 40003])
def test_words_follow_the_target(vocab):
    """Sums over the random numbers: over a fine grid of v the words of a row come as often as they weigh."""
    n = 4096
    g = torch.Generator().manual_seed(vocab)
    p = torch.softmax(2 * torch.randn(7, generator=g), -1)
    row = torch.zeros(vocab)
    place = torch.linspace(0, vocab - 1, 7).long()
    row[place] = p
    last = (torch.arange(n) + 0.5) / n
    z = torch.zeros(0)
    tokens, _ = lib().verify_draft(row.cuda().expand(n, vocab), z.int().cuda(), z.cuda(), last.cuda(),
                                   cu_draft=torch.zeros(n + 1, dtype=torch.int32, device="cuda"))
    often = torch.bincount(tokens.cpu().long(), minlength=vocab)[place] / n
    assert (often - p / p.sum()).abs().max() <= 1.0 / n  # each end of a word's run is off by half a step of the grid at most


def test_offsets_out_of_range():
    """Nothing outside of the buffers is read or written, whatever the offsets say."""
    s = _batch([2, 3, 1], 500, F32, 4)
    for cu in ([-5, 2, 100, 3], [0, 7, 2, 6], [6, 6, 6, 6], [2 ** 31 - 1, -2 ** 31, 0, 2 ** 31 - 1]):
        s["cu"] = torch.tensor(cu, dtype=torch.int32)
        got = _run(s)
        assert got[0].numel() == 9
    torch.cuda.synchronize()


def test_replays():
    """A captured call against eager ones over new probabilities, with other work between."""
    for vocab in (3001, 50001):
        s = _batch([3, 0, 5], vocab, F32, 2)
        d = {k: v.cuda() for k, v in s.items()}
        call = lambda: lib().verify_draft(d["target"], d["draft"], d["uniform"], d["last"], d["q"], d["cu"])  # noqa: E731
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for k in range(4):
            new = _batch([3, 0, 5], vocab, F32, 30 + k)
            for x in d:
                d[x].copy_(new[x])
            graph.replay()
            torch.cuda.synchronize()
            want = call()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            assert out[0].tolist() == do.verify(*(new[x] for x in ("target", "draft", "uniform", "last", "q", "cu")))[0]
