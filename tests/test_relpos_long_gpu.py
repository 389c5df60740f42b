"""The position bias at the largest sizes that it takes: positions whose byte offsets pass 32 bits."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

STARTS = (0, 1, 2, 3, 5, 8, 13, 21)


def rows_of(d):
    """The table's row of each difference (two-sided)."""
    n = d.abs()
    k = sum((n >= s).long() for s in STARTS[1:])
    return k + len(STARTS) * (d > 0).long()


@pytest.mark.parametrize("past", [0, 5, 2048])
def test_more_than_2_to_30_queries(past):
    """One key, 2^30 queries and some, whose positions differ from those 2^30 before. The table's entries are whole numbers that
    BF16 holds and so are the gradients, with sums below 2^24: everything is exact."""
    n = (1 << 30) + past
    gen = torch.Generator(device="cuda").manual_seed(past)
    pos = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    head, tail = slice(0, 3000), slice(n - 3000, n)
    for s in (head, tail):
        pos[0, s] = torch.randint(-30, 31, (3000,), generator=gen, device="cuda", dtype=torch.int32)
    key = torch.full((1, 1), 3, dtype=torch.int32, device="cuda")
    table = torch.arange(1, 17, device="cuda").float()[:, None]  # (numbers that BF16 holds)
    bias = tb.relpos_forward(table, STARTS, n, 1, positions=pos, key_positions=key).view(-1)
    for s in (head, tail):
        assert torch.equal(bias[s].float(), table[rows_of(3 - pos[0, s].long()), 0])
    middle = bias[4000:n - 4000]
    assert (middle.min() == middle.max()) and middle[0].item() == table[rows_of(torch.tensor(3)), 0].item()
    bias.zero_()
    at = torch.arange(n - 2900, n, 97, device="cuda")
    bias[at] = torch.arange(1, len(at) + 1, device="cuda").to(torch.bfloat16)  # (small whole numbers: every sum is exact)
    want = torch.zeros(16, dtype=torch.float64, device="cuda").index_add_(0, rows_of(3 - pos[0, at].long()), bias[at].double())
    got = tb.relpos_backward(bias.view(1, 1, n, 1), STARTS, positions=pos, key_positions=key)
    assert torch.equal(got[:, 0].double(), want)
