"""What probabilities weigh in the verification of drafts, those that are none among them, from the declaration alone: a
negative or NaN probability weighs nothing, in the target as in the drafter; and what a call writes, byte by byte."""
import ctypes
import math

import pytest
import torch

from gpu_support import lib
from test_gpu_verify_draft import BF16, F16, F32, _batch

pytestmark = pytest.mark.gpu


def _weighs(x):
    x = x.double()
    return torch.where(x > 0, x, 0.0)  # NaN is not above 0


def _declared(s):
    """(tokens, accepted) of each request by the declaration, in 64 bits."""
    tokens, accepted = [], []
    p_all, vocab = _weighs(s["target"]), s["target"].shape[1]
    for b in range(len(s["cu"]) - 1):
        t0, n = int(s["cu"][b]), int(s["cu"][b + 1] - s["cu"][b])
        rows = p_all[t0 + b:t0 + b + n + 1]
        kept, w = 0, None
        for i in range(n):
            d = int(s["draft"][t0 + i])
            q = torch.zeros(vocab, dtype=torch.float64)
            if s["q"] is not None:
                q = _weighs(s["q"][t0 + i])
            elif 0 <= d < vocab:
                q[d] = 1.0
            if 0 <= d < vocab and float(s["uniform"][t0 + i]) * float(q[d]) < float(rows[i, d]):
                kept += 1
                continue
            w = (rows[i] - q).clamp(min=0.0)
            if s["q"] is None:
                w = rows[i].clone()
                if 0 <= d < vocab:
                    w[d] = 0.0
            break
        if w is None or not float(w.sum()) > 0:
            w = rows[kept]
        upto = w.cumsum(0)
        word = int((upto > float(s["last"][b]) * upto[-1]).int().argmax()) if float(upto[-1]) > 0 else -1
        tokens += [int(x) for x in s["draft"][t0:t0 + kept]] + [word] + [-1] * (n - kept)
        accepted.append(kept)
    return tokens, accepted


def _run(s):
    d = {k: None if v is None else v.cuda() for k, v in s.items()}
    got = lib().verify_draft(d["target"], d["draft"], d["uniform"], d["last"], d["q"], d["cu"])
    return got[0].tolist(), got[1].tolist()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [500, 20001])
@pytest.mark.parametrize("certain", [False, True])
def test_no_probabilities_among_them(dtype, vocab, certain):
    """Negative numbers, -0, NaN and -inf in places of both."""
    for seed in range(4):
        s = _batch([3, 0, 5, 1, 2, 2], vocab, dtype, seed + vocab, certain=certain, far=2.0)
        g = torch.Generator().manual_seed(seed)
        for x in ("target", "q"):
            if s[x] is None:
                continue
            for bad in (-0.5, -0.0, math.nan, -math.inf):
                s[x][torch.rand(s[x].shape, generator=g) < 0.08] = bad
        assert _run(s) == _declared(s)


@pytest.mark.parametrize("vocab", [64, 20001])
def test_a_word_of_no_weight_is_not_drawn(vocab):
    """Where the target gives nothing or less, whatever the drafter says of the word."""
    s = _batch([1] * 6, vocab, F32, 3)
    s["target"][:] = 0.0
    s["target"][:, 7] = 1.0
    s["uniform"][:] = 0.5
    s["draft"][:] = 9
    s["q"][:] = 0.0
    for b, (p, q) in enumerate([(-0.1, -0.5), (0.0, -0.5), (-0.1, -math.inf), (0.0, math.nan), (math.nan, -0.5), (-0.2, -0.1)]):
        s["target"][2 * b, 3], s["q"][b, 3] = p, q      # a word that must not come out,
        s["target"][2 * b, 9], s["q"][b, 9] = p, q      # and a draft that must not stay
    for v in (0.0, 0.4, 1 - 2.0 ** -24):
        s["last"][:] = v
        got = _run(s)
        assert got[1] == [0] * 6
        assert got[0][::2] == [7] * 6
        assert got == _declared(s)


@pytest.mark.parametrize("vocab", [64, 20001])
def test_a_drafter_that_gave_a_draft_nothing(vocab):
    """A NaN or a negative number of the drafter's is 0: a draft that the target knows is kept."""
    s = _batch([1, 1, 1], vocab, F32, 4)
    s["uniform"][:] = 1 - 2.0 ** -24
    for b, q in enumerate((math.nan, -1.0, 0.0)):
        s["q"][b, int(s["draft"][b])] = q
    assert _run(s) == _declared(s) and _run(s)[1] == [1, 1, 1]


@pytest.mark.parametrize("vocab", [500, 20001])
@pytest.mark.parametrize("certain", [False, True])
def test_what_is_written(vocab, certain):
    """Whatever the offsets say, the outputs' own places and the workspace's, and nothing beside them."""
    from hashed_gram_memory_amd import serving as sv
    s = _batch([2, 3, 1], vocab, F32, 4, certain=certain)
    d = {k: None if v is None else v.cuda() for k, v in s.items()}
    n_seq, n_draft, mark = 3, 6, 64
    tokens = torch.full((mark + n_draft + n_seq + mark,), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    accepted = torch.full((mark + n_seq + mark,), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    for cu in ([0, 2, 5, 6], [-5, 2, 100, 3], [0, 7, 2, 6], [6, 6, 6, 6], [2 ** 31 - 1, -2 ** 31, 0, 2 ** 31 - 1], [3, 3, 6, 6]):
        tokens.fill_(0x5A5A5A5A)
        accepted.fill_(0x5A5A5A5A)
        offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        desc = sv.VerifyDraftDesc(target=d["target"].data_ptr(), draft_probs=0 if certain else d["q"].data_ptr(),
                                  draft=d["draft"].data_ptr(), uniform=d["uniform"].data_ptr(), last_uniform=d["last"].data_ptr(),
                                  cu_draft=offsets.data_ptr(), tokens=tokens[mark:].data_ptr(),
                                  n_accepted=accepted[mark:].data_ptr(), n_seq=n_seq, n_draft=n_draft, vocab=vocab,
                                  target_stride=vocab, draft_stride=0 if certain else vocab, type=sv.F32)
        need = ctypes.c_size_t()
        assert sv._lib.engram_verify_draft_workspace(ctypes.byref(desc), ctypes.byref(need)) == 0
        ws = torch.full((need.value + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        assert sv._lib.engram_verify_draft(ctypes.byref(desc), ws.data_ptr(), need.value, stream) == 0
        torch.cuda.synchronize()
        for x, n in ((tokens, n_draft + n_seq), (accepted, n_seq)):
            assert (x[:mark] == 0x5A5A5A5A).all() and (x[mark + n:] == 0x5A5A5A5A).all(), cu
        assert (ws[need.value:] == 0x5A).all(), cu
        got = accepted[mark:mark + n_seq].tolist()
        assert all(0 <= x <= n_draft for x in got), cu
        if cu == [0, 2, 5, 6]:
            assert (tokens[mark:mark + n_draft + n_seq].tolist(), got) == _declared(s)
