"""Shapes at which the kernels' loops go round many times on 152 SMs, against the 64-bit forms and with the tolerances
of test_norm_gpu.py (at most 60 rows a thread group in the column sums here) and test_cross_gpu.py."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from tests.test_cross_gpu import check, make
from tests.test_norm_gpu import _check_backward, _check_forward, _normal, _values, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,C,dtype", [
    (100000, 128, torch.float32),   # forward: CTAs that stay and load ahead, 7 trips; backward 28
    (20011, 512, torch.float32),    # four chunks a lane, loaded ahead, 8 trips; backward in pairs of rows, 17
    (6000, 1021, torch.bfloat16),   # the same with words shifted when used; rows in step
    (5001, 2048, torch.bfloat16),   # backward in pairs of rows, 9 trips, the last row alone
    (5000, 2048, torch.float32),
    (4003, 4000, torch.bfloat16),   # forward in CTAs of 128 threads, loaded ahead
    (4000, 4099, torch.float16),
    (2001, 8192, torch.bfloat16),
    (2000, 8192, torch.float32),
    (1501, 8190, torch.float32),    # rows that start on 8-byte boundaries
    (30000, 250, torch.bfloat16),
], ids=str)
def test_layer_norm(M, C, dtype):
    x, dy = _normal((M, C), dtype, 51), _normal((M, C), dtype, 52, 1.0, 0.0)
    gamma, beta = _weights(C, 53)
    y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_backward(x, gamma, mean, rstd, dy, tb.norm_backward(x, gamma, mean, rstd, dy))
    q, s, v = _values(x)
    assert torch.equal(kept.q8, q) and torch.equal(kept.scale, s)
    _check_backward(v, gamma, mean, rstd, dy, tb.norm_backward(kept, gamma, mean, rstd, dy))


@pytest.mark.parametrize("M,C,width", [(20000, 96, 104), (6000, 1000, 1021)])
def test_layer_norm_of_spaced_rows(M, C, width):
    x, dy = _normal((M, width), torch.bfloat16, 54)[:, 4:4 + C], _normal((M, width), torch.bfloat16, 55, 1.0, 0.0)[:, 4:4 + C]
    gamma, beta = _weights(C, 56)
    y, mean, rstd = tb.norm_forward(x, gamma, beta)
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_backward(x, gamma, mean, rstd, dy, tb.norm_backward(x, gamma, mean, rstd, dy))


@pytest.mark.parametrize("B,T,S,H,Hk,d,lens,mask", [
    (2, 1100, 2000, 16, 16, 128, None, None),            # forward 17 units a CTA, whole runs one behind another; backward 30
    (2, 1100, 2000, 16, 16, 64, None, None),
    (2, 1100, 2000, 16, 4, 128, [2000, 1333], 0.9),      # the same with masked keys to be zeroed in every tile
    (2, 1100, 2000, 8, 8, 40, [1999, 1200], None),
    (64, 300, 100, 16, 16, 128, None, None),             # runs of one unit, two row tiles and one in turn
    (40, 512, 100, 16, 16, 128, None, None),             # runs of one unit, always two row tiles
    (40, 512, 128, 16, 16, 64, [128, 0, 1, 77], None),
    (24, 512, 250, 16, 8, 128, [250, 17, 128, 0], 0.8),  # runs of one and two units
    (3, 100, 4000, 16, 16, 128, None, None),             # one row tile: even and odd key tiles as streams
    (1, 3000, 300, 12, 4, 96, None, None),               # key tiles with many row tiles, groups of three
    (16, 3, 3000, 28, 4, 128, None, None),               # groups of seven
], ids=str)
def test_cross_attention(B, T, S, H, Hk, d, lens, mask):
    x = make(B, T, S, H, Hk, d, lens=lens, mask=mask, seed=21)
    first = check(x)
    for _ in range(3):
        O, LSE = tb.cross_forward(x["q"], x["k"], x["v"], x["mask"], x["lens"])
        again = (O, LSE, *tb.cross_backward(x["q"], x["k"], x["v"], O, LSE, x["do"], x["mask"], x["lens"]))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert tb.tri_attn_device_status() == 0
