"""The relative position bias and its gradient (include/tri_relpos.h) against the definition, with the buckets in whole
numbers on the host.

Tolerances: the forward adds two numbers in FP32 and rounds once (2^-8 |result| + 2^-23 of the magnitudes); the
gradient is an FP32 sum of numbers of BF16: a lane adds under 2^13 of them in turn here, then trees and under 2^8 partial
sums: 2^13 x 2^-24 of the sum of magnitudes at the worst, F = 2^-11.
"""
import bisect

import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

F = 2.0 ** -11
LOG16 = tb.relpos_starts(32, 128)
CASES = [  # B, H, Nq, Nk, starts, two-sided
    (1, 1, 1, 1, (0,), True), (1, 1, 1, 1, (0, 1), False), (2, 3, 7, 5, (0, 1, 2), True), (1, 4, 33, 100, LOG16, True),
    (2, 2, 100, 33, LOG16, False), (1, 2, 129, 131, tuple(range(33)), True), (1, 3, 1, 1003, LOG16, True), (3, 1, 1003, 1, LOG16, False),
    (1, 16, 384, 384, LOG16, True), (2, 2, 300, 301, (0, 5, 9), True), (1, 2, 200, 6000, (0, 1, 50, 4096), True),
    (1, 2, 200, 6000, (0, 1, 50, 4097), True), (1, 1, 50, 9000, (0, 3, 5000, 8000), False), (1, 2, 64, 64, tuple(range(128)), True),
    (1, 1, 40, 5000, tuple(40 * k for k in range(128)), True), (1, 2, 40, 40, (0,), False), (1, 2, 40, 40, (0,), True),
    (2, 9, 61, 63, LOG16, True), (3, 8, 50, 70, LOG16, False), (1, 10, 33, 31, (0,), False), (1, 8, 100, 101, (0, 2), True),
    (1, 8, 30, 4000, tuple(40 * k for k in range(128)), True), (2, 8, 1, 1, (0, 1), True), (2, 9, 3, 1, LOG16, True),
    (2, 8, 1, 5, LOG16, False), (3, 8, 2, 3, (0, 2), True), (1, 9, 700, 2, LOG16, True)]


def rows_of(starts, two, q, k):
    """[Nq, Nk] rows of the table, from whole numbers on the host."""
    K, d = len(starts), k[None, :].cpu().long() - q[:, None].cpu().long()
    n = d.abs() if two else (-d).clamp(min=0)
    at = torch.searchsorted(torch.tensor(starts), n, right=True) - 1
    return (at + K * (d > 0) if two else at).cuda()


def test_rows_of_one_by_one():
    q, k = torch.arange(9), torch.arange(13) * 3 - 7
    rows = rows_of(LOG16, True, q, k)
    for i in range(9):
        for j in range(13):
            d = int(k[j] - q[i])
            assert rows[i, j] == bisect.bisect_right(LOG16, abs(d)) - 1 + (16 if d > 0 else 0)


def check(B, H, Nq, Nk, starts, two, positions, key_positions, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R = len(starts) * (2 if two else 1)
    table = torch.randn((R, H), generator=gen, device="cuda")
    base, dbias = (torch.randn((B, H, Nq, Nk), generator=gen, device="cuda").bfloat16() for _ in range(2))
    kw = dict(positions=positions, key_positions=key_positions, two_sided=two)
    plain = tb.relpos_forward(table, starts, Nq, Nk, B=B, **kw)
    onto = tb.relpos_forward(table, starts, Nq, Nk, B=B, base=base, **kw)
    dtable = tb.relpos_backward(dbias, starts, **kw)
    assert dtable.shape == (R, H)
    want, mag = torch.zeros((R, H), dtype=torch.float64, device="cuda"), torch.zeros((R, H), dtype=torch.float64, device="cuda")
    for b in range(B):
        q = torch.arange(Nq) if positions is None else positions[b]
        k = torch.arange(Nk) if positions is None else (positions if key_positions is None else key_positions)[b]
        rows = rows_of(starts, two, q, k)
        t = table.double()[rows].permute(2, 0, 1)
        assert torch.equal(plain[b], table[rows].permute(2, 0, 1).bfloat16())
        w = t + base[b].double()
        assert ((onto[b].double() - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -23 * (t.abs() + base[b].double().abs())).all()
        d = dbias[b].double().permute(1, 2, 0).reshape(-1, H)
        want.index_add_(0, rows.flatten(), d)
        mag.index_add_(0, rows.flatten(), d.abs())
    assert ((dtable.double() - want).abs() <= F * mag).all()
    assert torch.equal(dtable, tb.relpos_backward(dbias, starts, **kw))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, (*c[:4], len(c[4]), c[4][-1], c[5]))))
def test_forward_and_backward(case):
    check(*case, None, None)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, (*c[:4], len(c[4]), c[4][-1], c[5]))))
def test_positions(case):
    B, H, Nq, Nk, starts, two = case
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randint(-500, 5000, (B, Nq), generator=gen, device="cuda", dtype=torch.int32)
    k = torch.randint(-500, 5000, (B, Nk), generator=gen, device="cuda", dtype=torch.int32)
    check(*case, q, k)
    if Nq == Nk:
        check(*case, q, None)


def test_positions_at_the_ends_of_their_type():
    ends = torch.tensor([[-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    for starts in ((0,), (0, 1, 2), (0, 1, 2 ** 31 - 1), (0, 5, 2 ** 30)):
        for two in (True, False):
            table = torch.randn((len(starts) * (2 if two else 1), 2), device="cuda")
            got = tb.relpos_forward(table, starts, 6, positions=ends, two_sided=two)
            d = (ends[:, None, :].long() - ends[:, :, None].long()).clamp(-2 ** 31 + 1, 2 ** 31 - 1)[0]
            n = d.abs() if two else (-d).clamp(min=0)
            rows = torch.searchsorted(torch.tensor(starts).cuda(), n, right=True) - 1 + (len(starts) * (d > 0) if two else 0)
            assert torch.equal(got[0], table[rows].permute(2, 0, 1).bfloat16())


def test_in_place_on_the_pair_bias():
    base = torch.randn((1, 4, 77, 77), device="cuda").bfloat16()
    table = torch.randn((32, 4), device="cuda")
    want = tb.relpos_forward(table, LOG16, 77, base=base)
    shape = tb.RelposShape(1, 4, 77, 77, 16, 1)
    tb.tri_relpos_fwd(shape, LOG16, table, None, None, base, base)
    assert torch.equal(base, want)


def test_many_planes():
    """More planes than one axis of a grid, and pieces that all heads share."""
    check(40000, 1, 3, 5, (0, 1, 2), True, None, None)
