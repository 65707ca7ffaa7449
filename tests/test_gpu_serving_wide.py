"""Chunks divide their keys by what the requests hold, not by how wide the table is: the same bits."""
import pytest
import torch

from test_gpu_serving import BF16, F16, _attend, _paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,e4m3,D,H,new,lens", [
    (BF16, False, 128, 1, [64], [4096]),
    (F16, False, 64, 2, [40], [3900]),
    (BF16, True, 256, 1, [90], [2500]),
    (BF16, False, 128, 2, [300], [2048]),
    (F16, True, 64, 1, [20, 90, 1, 5, 0], [4096, 700, 333, 90, 3000]),  # with requests of few rows, some longer, and of none
], ids=str)
def test_the_table_s_width(dtype, e4m3, D, H, new, lens):
    s = _paged(sum(new) + D, dtype, e4m3, D, H, 4, 16, new, lens)
    near = _attend(s, max_q_len=max(new))
    for width in (2000, 8192):
        wide = torch.full((len(new), width), -1, dtype=torch.int32)
        wide[:, :s["table"].shape[1]] = s["table"]
        far = _attend(dict(s, table=wide), max_q_len=max(new))
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_a_long_request_of_one_token_beside_a_chunk():
    """The lengths that count are those of the requests with many rows: the chunk's bits are those it has alone."""
    s = _paged(5, BF16, False, 128, 1, 4, 16, [64, 1], [4096, 30000])
    both = _attend(s, max_q_len=64)
    alone = _attend(dict(s, q=s["q"][:64], table=s["table"][:1], kv_len=s["kv_len"][:1], equal=True))
    assert torch.equal(both[0][:64], alone[0]) and torch.equal(both[1][:64], alone[1])
