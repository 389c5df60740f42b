"""The feed-forward block's one-kernel forward while other work takes memory's time: the order in which its copies land
differs from call to call, its results do not."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from tests.test_ffn_gpu import check_forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,C,Fh,keep", [(147456, 128, 512, False), (60000, 64, 200, True), (39000, 8, 72, False), (58400, 200, 264, False)])
def test_the_same_bits_beside_other_work(M, C, Fh, keep):
    x, wg, wu, wd, _ = inputs(M, C, Fh, 4)
    first = tb.ffn_forward(x, wg, wu, wd, keep=True)
    check_forward(x, wg, wu, wd, "silu", *first)
    other, a = torch.cuda.Stream(), torch.randn(1 << 26, device="cuda")
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for n in range(40):
        with torch.cuda.stream(other):
            for k in range(n % 4):
                b.copy_(a)
                a[:1 << 20].mul_(1.0)
        for k in range(3):
            got = tb.ffn_forward(x, wg, wu, wd, keep=keep)
            assert all(torch.equal(p, q) for p, q in zip(first, got if keep else (got,)))
    other.synchronize()
    assert tb.tri_attn_device_status() == 0
