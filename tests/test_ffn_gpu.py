"""The gated feed-forward block (include/tri_ffn.h) against its formulas in 64 bits.

Tolerances, from the arithmetic. U = 2^-8 is half a step of BF16, relative. An output is a sum of n products of a
rounded operand (h, da or du: off by at most U each, and by the activation's FP32 error, a few 2^-22, below) with an
exact one, added in FP32 (sums of at most 2^15 terms here, in blocks of 16 inside the tensor cores: under 2^12
roundings or cut-offs of 2^-23, and usually far less: F = 2^-11), then rounded once: |error| <= U |result| + (U + F) sum |products|.
a and u have exact operands: U |result| + F sum |products|. h in the backward pass is formed from the kept, rounded a
and u, and so is the oracle's. erff's own bound is 2 ulp; 1 + erf cancels for negative a, which the absolute error
2^-22 |a u| of h covers: small against U times the magnitudes, as sums of products with |h| near its size show, but
not element by element, so every product counts |h| + 2^-20 |a u| in the sum of magnitudes.
"""
import math

import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -11
ACTS = ["silu", "gelu", "sigmoid"]
# (rows, channels, features): tiles filled and not, one row, one block of channels, shares of a tile over many pairs
SIZES = [(1, 8, 8), (1, 64, 128), (7, 72, 200), (128, 64, 64), (129, 128, 512), (256, 256, 256), (300, 136, 1032), (513, 384, 1536),
         (1000, 264, 264), (4001, 392, 1032), (9, 2048, 8192), (20000, 128, 512), (64, 4096, 520),
         (19500, 64, 200), (39999, 200, 264), (60001, 256, 64), (19457, 8, 8), (50000, 136, 328), (80000, 128, 64),
         (2, 1000, 3000), (8, 4096, 1032), (15, 264, 72), (16, 2048, 520), (17, 72, 4104), (31, 520, 264), (32, 1032, 2048), (33, 1032, 2048),
         (10000, 1032, 2056), (150000, 72, 64), (150001, 128, 48), (100000, 200, 40), (120000, 128, 72), (99999, 256, 136)]


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()


def inputs(M, C, Fh, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (normal(gen, M, C), normal(gen, Fh, C, std=C ** -0.5), normal(gen, Fh, C, std=C ** -0.5),
            normal(gen, C, Fh, std=Fh ** -0.5), normal(gen, M, C))


def act64(a, act):
    """act(a) and its derivative."""
    if act == "gelu":
        phi = 0.5 * torch.erfc(-a * math.sqrt(0.5))
        return a * phi, phi + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(a)
    return (a * s, s * (1 + a * (1 - s))) if act == "silu" else (s, s * (1 - s))


def close(got, want, mag, operand=U, out=U):
    assert got.isfinite().all()
    err = (got.double() - want).abs()
    tol = out * want.abs() + (operand + F) * mag
    assert (err <= tol).all(), f"{(err / tol).max().item()} of the tolerance, {(err > tol).sum().item()} places"


def check_forward(x, wg, wu, wd, act, out, a, u):
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    a64, u64 = x @ wg.T, x @ wu.T
    if a is not None:
        close(a, a64, x.abs() @ wg.abs().T, 0.0)
        close(u, u64, x.abs() @ wu.abs().T, 0.0)
    h = act64(a64, act)[0] * u64
    # (FP32 sums behind a and u: at most F of their magnitudes through act's slope, at most 1.13, and u)
    da, du = F * (x.abs() @ wg.abs().T), F * (x.abs() @ wu.abs().T)
    mag = h.abs() + 2.0 ** -20 * (a64 * u64).abs() + (1.2 * da * u64.abs() + act64(a64, act)[0].abs() * du) / U
    close(out, h @ wd.T, mag @ wd.abs().T)


def check_backward(x, wg, wu, wd, a, u, dout, act, got, out=U):
    x, wg, wu, wd, a, u, dout = (t.double() for t in (x, wg, wu, wd, a, u, dout))
    f, df = act64(a, act)
    dh, mh = dout @ wd, F * (dout.abs() @ wd.abs())
    da, du, h = dh * u * df, dh * f, f * u
    ma = da.abs() + (mh * (u * df).abs() + 2.0 ** -20 * (dh * u).abs() * (1 + a.abs())) / U
    mu = du.abs() + (mh * f.abs() + 2.0 ** -20 * (dh * a).abs()) / U
    mw = h.abs() + 2.0 ** -20 * (a * u).abs() / U
    dx, dwg, dwu, dwd = got
    if dx is not None:
        close(dx, da @ wg + du @ wu, ma @ wg.abs() + mu @ wu.abs())
    if dwg is not None:
        close(dwg, da.T @ x, ma.T @ x.abs(), out=out)
        close(dwu, du.T @ x, mu.T @ x.abs(), out=out)
        close(dwd, dout.T @ h, dout.abs().T @ mw, out=out)


@pytest.mark.parametrize("M,C,Fh", SIZES)
def test_forward_and_backward(M, C, Fh):
    act = ACTS[(M + C + Fh) % 3]
    x, wg, wu, wd, dout = inputs(M, C, Fh)
    out, a, u = tb.ffn_forward(x, wg, wu, wd, act=act, keep=True)
    assert tb.tri_attn_device_status() == 0
    check_forward(x, wg, wu, wd, act, out, a, u)
    assert torch.equal(out, tb.ffn_forward(x, wg, wu, wd, act=act))
    got = tb.ffn_backward(x, wg, wu, wd, a, u, dout, act=act)
    assert tb.tri_attn_device_status() == 0
    check_backward(x, wg, wu, wd, a, u, dout, act, got)


@pytest.mark.parametrize("M,C,Fh", [(1, 8, 8), (300, 136, 1032), (2000, 72, 40), (5000, 264, 520)])
def test_weight_gradients_in_32_bits(M, C, Fh):
    """Their own rounding is FP32's: what is left is that of h, da and du."""
    x, wg, wu, wd, dout = inputs(M, C, Fh, 2)
    _, a, u = tb.ffn_forward(x, wg, wu, wd, keep=True)
    got = tb.ffn_backward(x, wg, wu, wd, a, u, dout, weight_dtype=torch.float32)
    assert all(t.dtype == torch.float32 for t in got[1:])
    check_backward(x, wg, wu, wd, a, u, dout, "silu", got, out=2.0 ** -24)
    some = tb.ffn_backward(x, wg, wu, wd, a, u, dout, need_dw=False)
    assert torch.equal(some[0], got[0]) and some[1:] == (None, None, None)
    some = tb.ffn_backward(x, wg, wu, wd, a, u, dout, need_dx=False, weight_dtype=torch.float32)
    assert some[0] is None and all(torch.equal(p, q) for p, q in zip(some[1:], got[1:]))


@pytest.mark.parametrize("M,C,Fh", [(5, 128, 256), (100, 72, 200), (20000, 64, 128)])
def test_projections_alone(M, C, Fh):
    """What a pass that recomputes them asks for: the bits of the whole forward, in each of its forms but the one kernel's,
    whose sums run in the same order too."""
    x, wg, wu, wd, _ = inputs(M, C, Fh, 3)
    _, a, u = tb.ffn_forward(x, wg, wu, wd, keep=True)
    a2, u2 = tb.ffn_forward(x, wg, wu, wd, keep="only")
    assert torch.equal(a, a2) and torch.equal(u, u2)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 200, 20000])
def test_activations_far_out(act, M):
    """Gates from -1e30 to 1e30 (sums of one product each): finite, and as the formulas have it."""
    C = Fh = 64
    gates = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1.0, -1.0, -20.0, -39.0, -41.0, -80.0, -87.0, -88.0, -89.0, -120.0, -1e4, -1e30, 20.0, 89.0, 1e4, 1e30])
    x = torch.zeros(M, C, device="cuda")
    x[:, 0] = 1.0
    x = x.bfloat16()
    wg, wu = torch.zeros(Fh, C, device="cuda"), torch.zeros(Fh, C, device="cuda")
    wg[:, 0] = gates.repeat(4)[:Fh].cuda()
    wu[:, 0] = 2.0
    wg, wu, wd = wg.bfloat16(), wu.bfloat16(), torch.eye(Fh, device="cuda").bfloat16()
    out, a, u = tb.ffn_forward(x, wg, wu, wd, act=act, keep=True)
    f, df = act64(a[0].double(), act)
    assert torch.equal(a[0], wg[:, 0]) and ((out.double() - 2 * f).abs() <= 3 * U * (2 * f).abs() + 2.0 ** -19 * (1 + a[0].double().abs().clamp(max=6))).all()
    dx, dwg, dwu, _ = tb.ffn_backward(x, wg, wu, wd, a, u, x, act=act)
    assert dx.isfinite().all() and dwg.isfinite().all() and dwu.isfinite().all()
    want = M * 2 * df[0]  # (dout = x reaches feature 0 alone)
    assert abs(dwg[0, 0].item() - want.item()) <= 3 * U * abs(want.item()) + M * 2.0 ** -18
