"""Shapes at which the kernels' loops go round many times on 152 SMs, against the 64-bit forms and with the tolerances
of test_norm_gpu.py (at most 60 rows a thread group in the column sums here) and test_cross_gpu.py."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from tests.test_cross_gpu import check, close, make, oracle
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


@pytest.mark.parametrize("M,C", [(16777224, 136), (16777224, 135)])
def test_layer_norm_offsets_past_32_bits(M, C):
    """More than 2^31 elements: rows at the ends and on either side of 2^31 elements have the bits that they have
    in calls on them alone; the weights' gradients are the sums of those of parts."""
    gen = torch.Generator(device="cuda").manual_seed(57)
    x, dy = (torch.empty((M, C), dtype=torch.bfloat16, device="cuda").normal_(0.25, 1.5, generator=gen) for _ in range(2))
    gamma, beta = _weights(C, 58)
    y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
    packed = tb.checkpoint_pack(x)
    dx, dgamma, dbeta = tb.norm_backward(x, gamma, mean, rstd, dy)
    dx8, _, _ = tb.norm_backward(kept, gamma, mean, rstd, dy)
    back = tb.checkpoint_unpack(packed)
    for a in (0, 2 ** 31 // C // 8 * 8 - 64, M - 128):
        s = slice(a, a + 128)
        y1, mean1, rstd1, kept1 = tb.norm_forward(x[s], gamma, beta, checkpoint=True)
        assert torch.equal(y[s], y1) and torch.equal(mean[s], mean1) and torch.equal(rstd[s], rstd1)
        for k in (kept, packed):
            assert torch.equal(k.q8[s], kept1.q8) and torch.equal(k.scale[s], kept1.scale)
        assert torch.equal(back[s], tb.checkpoint_unpack(kept1))
        assert torch.equal(dx[s], tb.norm_backward(x[s], gamma, mean1, rstd1, dy[s])[0])
        assert torch.equal(dx8[s], tb.norm_backward(kept1, gamma, mean1, rstd1, dy[s])[0])
    want, mag = [torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(2)], [0.0, 0.0]
    rows, step = 0, 1 << 20
    for a in range(0, M, step):
        xh, d = (x[a:a + step].float() - mean[a:a + step, None]) * rstd[a:a + step, None], dy[a:a + step].float()
        want[0] += (d.double() * xh.double()).sum(0)
        want[1] += d.double().sum(0)
        mag[0] = mag[0] + (d * xh).abs().double().sum(0)
        mag[1] = mag[1] + d.abs().double().sum(0)
        rows += d.shape[0]
    # 456 CTAs of 36800 rows in eight lane groups (17 or 18 chunks in 32 lanes): 4600 roundings in turn, then trees: 2^-11
    assert rows == M
    for got, w, m in zip((dgamma, dbeta), want, mag):
        assert ((got.double() - w).abs() <= 2.0 ** -11 * m).all()


def test_cross_attention_with_the_most_queries():
    """2^26 queries: rows at the ends and in the middle have the bits of calls on them alone."""
    T, S, d = 2 ** 26, 5, 8
    x = make(1, 1, S, 1, 1, d, seed=22)
    q, do = (torch.empty((1, T, 1, d), dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    O, LSE = tb.cross_forward(q, x["k"], x["v"])
    dQ, dK, dV = tb.cross_backward(q, x["k"], x["v"], O, LSE, do)
    for a in (0, T // 2 - 64, T - 128):
        s = slice(a, a + 128)
        O1, LSE1 = tb.cross_forward(q[:, s], x["k"], x["v"])
        assert torch.equal(O[:, s], O1) and torch.equal(LSE[..., s], LSE1)
        assert torch.equal(dQ[:, s], tb.cross_backward(q[:, s], x["k"], x["v"], O1, LSE1, do[:, s].contiguous())[0])
    # dV: sums over the queries, P rounded to BF16 and once more at the end
    want, mag = 0.0, 0.0
    for a in range(0, T, 1 << 22):
        p = torch.exp(q[0, a:a + (1 << 22), 0].double() @ x["k"][0, :, 0].double().T * d ** -0.5 - LSE[0, 0, a:a + (1 << 22), None].double())
        g = do[0, a:a + (1 << 22), 0].double()
        want, mag = want + p.T @ g, mag + p.T @ g.abs()
    assert ((dV[0, :, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * mag).all()
    assert dK.isfinite().all() and tb.tri_attn_device_status() == 0


def test_cross_attention_with_the_most_keys():
    """2^26 keys of which a mask leaves a few, at the ends, in the middle and at tiles' edges."""
    S, d = 2 ** 26, 8
    k, v = (torch.empty((1, S, 1, d), dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    x = make(1, 3, 1, 1, 1, d, seed=23)
    keep = torch.tensor([0, 127, 128, S // 2 - 1, S // 2, S - 129, S - 1], device="cuda")
    mask = torch.zeros((1, S), dtype=torch.bool, device="cuda")
    mask[0, keep] = True
    O, LSE = tb.cross_forward(x["q"], k, v, mask)
    grads = tb.cross_backward(x["q"], k, v, O, LSE, x["do"], mask)
    few = dict(x, k=k[:, keep].contiguous(), v=v[:, keep].contiguous())
    for name, w in oracle(few, d ** -0.5).items():
        close(name, O if name == "O" else LSE, w, name == "O")
    ref = oracle(few, d ** -0.5, O, LSE)
    for name, g in zip(("dQ", "dK", "dV"), grads):
        close(name, g if name == "dQ" else g[:, keep], ref[name])
        if name != "dQ":
            assert torch.count_nonzero(g) <= keep.numel() * d
    assert tb.tri_attn_device_status() == 0
