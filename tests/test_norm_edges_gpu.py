"""LayerNorm (include/tri_norm.h) at the ends of its range, against the formulas in 64 bits. Tolerances as in
test_norm_gpu.py: half a step of the output's type, and F = 2^-17 of the magnitudes that enter an output for the FP32
arithmetic."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from tests.test_norm_gpu import F, _normal, _u, _values, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("M,C", [(3, 8), (9, 5), (30, 121), (33, 96), (20, 1000), (40, 1003), (12, 2040), (24, 4001), (17, 8190)])
def test_backward_of_constant_rows_far_from_zero(M, C, dtype, eight_bits):
    """|mean| rstd passes the largest FP32 number and every (x - mean) is 0: dx = rstd (g - sum(g) / C), dgamma = 0.
    What stands outside the row (lanes past its end, the tail of its last chunk, its neighbours in memory) has no part
    in it. The mean is the value that the row's elements have, so that the differences are 0 exactly: 127 x 2^117, whose
    checkpoint's scale 2^117 makes q s exact too (with 2e37, q s - mean would be the rounding of q s to 32 bits, up to
    2^99.2 = 7e29, whose square times rstd cubed is far beyond BF16 and FP32: the formula's own dx is)."""
    x = torch.full((M, C), 127 * 2.0 ** 117, dtype=dtype, device="cuda")
    dy, gamma = _normal((M, C), dtype, 41, 1.0, 0.0), _weights(C, 42)[0]
    given, values = x, x.float()
    if eight_bits:
        given = tb.checkpoint_pack(x)
        values = tb.checkpoint_unpack(given, torch.float32)
    mean, rstd = values[:, 0].contiguous(), torch.full((M,), 1e-5 ** -0.5, device="cuda")
    assert (values == mean[:, None]).all() and (mean * rstd).isinf().all()
    dx, dgamma, dbeta = tb.norm_backward(given, gamma, mean, rstd, dy)
    g, rs = dy.double() * gamma.double(), rstd.double()[:, None]
    want = rs * (g - g.mean(-1, keepdim=True))
    mag = rs * (g.abs() + g.abs().mean(-1, keepdim=True))
    assert ((dx.double() - want).abs() <= _u(dtype) * want.abs() + 2 * F * mag).all()
    assert (dgamma == 0).all()
    assert ((dbeta.double() - dy.double().sum(0)).abs() <= 2 * F * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("M,C,dtype", [(1, 2 ** 31 - 128, torch.bfloat16), (3, 2 ** 29 + 5, torch.float16)], ids=str)
def test_checkpoints_of_the_widest_rows(M, C, dtype):
    """Rows of billions of channels, checked group by group at their ends and on either side of 2^31 bytes."""
    x = torch.empty((M, C), dtype=dtype, device="cuda").normal_()
    kept = tb.checkpoint_pack(x)
    back = tb.checkpoint_unpack(kept, dtype)
    assert kept.scale.shape == (M, (C + 127) // 128)
    for m in range(M):
        for g in (0, 2 ** 22 - 64, 2 ** 23 - 64, 2 ** 24 - 2 ** 10, (C - 1) // 128 - 63):
            a, b = 128 * g, min(128 * (g + 64), C)
            if a >= C:
                continue
            q, s, v = _values(x[m:m + 1, a:b])
            assert torch.equal(kept.q8[m:m + 1, a:b], q) and torch.equal(kept.scale[m:m + 1, g:g + s.shape[1]], s)
            assert torch.equal(back[m:m + 1, a:b], v.to(dtype))
