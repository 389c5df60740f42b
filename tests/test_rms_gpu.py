"""RMS norm with a residual and an 8-bit output (include/tri_rms.h) against plain 64-bit forms.

Tolerances, from the arithmetic. u is half a step of the output type (torch.finfo(t).eps / 2): one rounding of the
result; below the type's smallest normal number the step is that of the smallest one, s = smallest_normal x eps, whatever
the value (FP16: 2^-24, which a y of 0.00001 meets), so half of s comes to it. The rest is FP32: a row's sum is at most 8 chunks of 8 values in turn, a shuffle tree and 8 warps (under 128
roundings of 2^-24, relative to the sum of magnitudes), a handful of operations follow: F = 2^-17 times the magnitudes
that enter an output. A column sum adds a chunk of rows in turn (under 100 in these tests) and then trees: the same.
r is exact: the FP32 sum of two numbers of the type, rounded (for 16-bit types that sum is itself rounded where the exponents are
over 13 apart; the oracle does the same). The 8-bit output's scale is FP32 of the row's FP32 values: its values are
off by half a step of the group, top / 254, and F.
"""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

F = 2.0 ** -17
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [(1, 1), (5, 1), (1, 8), (3, 5), (7, 64), (33, 128), (100, 130), (17, 256), (9, 384), (40, 512), (64, 768),
         (5, 1003), (3, 1024), (12, 2048), (5, 4099), (2, 8192), (3, 8191), (2000, 16), (50, 27), (61, 59), (40, 121),
         (300, 30), (700, 1003), (150, 4001), (77, 259), (3000, 128)]


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _normal(shape, dtype, seed, std=1.5, mean=0.25):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _check_forward(x, residual, gamma, eps, got):
    r = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    if residual is None:
        assert got.r is None
    else:
        assert torch.equal(got.r, r)
    rd = r.double()
    rstd = 1.0 / torch.sqrt((rd * rd).mean(-1) + eps)
    assert got.rstd.dtype == torch.float32 and got.rstd.shape == x.shape[:-1]
    assert ((got.rstd.double() - rstd).abs() <= F * rstd).all()
    want = rd * rstd[..., None] * (1.0 if gamma is None else gamma.double())
    if got.y is not None:
        assert got.y.dtype == x.dtype and got.y.shape == x.shape and got.y.is_contiguous()
        assert ((got.y.double() - want).abs() <= (_u(x.dtype) + 2 * F) * want.abs() + _least(x.dtype)).all()
    if got.y8 is not None:
        C = x.shape[-1]
        n = (C + 127) // 128
        top = torch.nn.functional.pad(want.abs(), (0, n * 128 - C)).unflatten(-1, (n, 128)).amax(-1)
        assert got.y8.scale.shape == top.shape and ((got.y8.scale.double() - top / 127).abs() <= 2 * F * top / 127).all()
        step = (top / 127).repeat_interleave(128, -1)[..., :C]
        values = got.y8.q8.double() * got.y8.scale.double().repeat_interleave(128, -1)[..., :C]
        assert ((values - want).abs() <= step * (0.5 + 128 * 4 * F)).all()
        assert torch.equal(tb.checkpoint_unpack(got.y8, torch.float32).double(), (got.y8.q8.float() * got.y8.scale.repeat_interleave(128, -1)[..., :C]).double())


def _check_backward(r, gamma, rstd, dy, dr, got):
    rd, d, rs = r.double(), dy.double(), rstd.double()[..., None]
    g = d if gamma is None else d * gamma.double()
    rh = rd * rs
    dx = rs * (g - rh * (g * rh).mean(-1, keepdim=True))
    mag = rs * (g.abs() + rh.abs() * (g * rh).abs().mean(-1, keepdim=True))
    if dr is not None:
        dx, mag = dx + dr.double(), mag + dr.double().abs()
    assert got[0].dtype == dy.dtype and got[0].shape == dy.shape
    assert ((got[0].double() - dx).abs() <= _u(dy.dtype) * dx.abs() + 2 * F * mag + _least(dy.dtype)).all()
    if gamma is None:
        assert got[1] is None
    else:
        rows = tuple(range(r.dim() - 1))
        assert ((got[1].double() - (d * rh).sum(rows)).abs() <= 2 * F * (d * rh).abs().sum(rows)).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,C", SIZES)
def test_forward_and_backward(M, C, dtype):
    x, res, dy, dr = (_normal((M, C), dtype, s) for s in (1, 2, 3, 4))
    gamma = _normal((C,), torch.float32, 5, 0.3, 1.0)
    for residual, past in ((res, dr), (None, None)):
        got = tb.rms_forward(x, gamma, residual, eight_bits=True)
        _check_forward(x, residual, gamma, 1e-5, got)
        only = tb.rms_forward(x, gamma, residual, eight_bits="only")
        assert only.y is None and torch.equal(only.y8.q8, got.y8.q8) and torch.equal(only.y8.scale, got.y8.scale)
        plain = tb.rms_forward(x, gamma, residual)
        assert plain.y8 is None
        _check_forward(x, residual, gamma, 1e-5, plain)  # (rows of odd width without the 8-bit output are added in another order)
        r = x if residual is None else got.r
        _check_backward(r, gamma, got.rstd, dy, past, tb.rms_backward(r, gamma, got.rstd, dy, past))


def test_without_weights():
    x, dy = _normal((37, 96), torch.bfloat16, 5), _normal((37, 96), torch.bfloat16, 6)
    got = tb.rms_forward(x, eight_bits=True)
    _check_forward(x, None, None, 1e-5, got)
    _check_backward(x, None, got.rstd, dy, None, tb.rms_backward(x, None, got.rstd, dy))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("C,width,start", [(128, 160, 16), (128, 160, 3), (100, 101, 0), (1000, 2048, 1)])
def test_spaced_and_unaligned_rows(C, width, start, dtype):
    """Rows that are part of wider ones (row strides, starts off the 16-byte boundaries), of a 3-D tensor."""
    x, res, dy, dr = (_normal((4, 9, width), dtype, s)[..., start:start + C] for s in (8, 9, 10, 11))
    gamma = _normal((C + 1,), torch.float32, 12, 0.3, 1.0)[1:]  # 4-byte alignment only
    got = tb.rms_forward(x, gamma, res, eight_bits=True)
    _check_forward(x, res, gamma, 1e-5, got)
    _check_backward(got.r, gamma, got.rstd, dy, dr, tb.rms_backward(got.r, gamma, got.rstd, dy, dr))
    _check_backward(x, gamma, got.rstd, dy, dr, tb.rms_backward(x, gamma, got.rstd, dy, dr))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("M,C,off", [(50, 259, 3), (9, 64, 1), (300, 1001, 2)])
def test_into_buffers_equally_far_from_a_boundary(M, C, off, dtype):
    """Buffers that start the same number of values behind a 16-byte boundary; nothing is written before or behind them."""
    vec = 128 // torch.finfo(dtype).bits
    wide = [torch.full((M * C + 2 * vec,), 7, dtype=dtype, device="cuda") for _ in range(6)]
    x, dy, dr, dx, r, y = (w[off:off + M * C].view(M, C) for w in wide)
    for s, t in enumerate((x, dy, dr)):
        t.copy_(_normal((M, C), dtype, 20 + s))
    gamma = _normal((C,), torch.float32, 22, 0.3, 1.0)
    rstd, dgamma = torch.empty(M, device="cuda"), torch.empty(C, device="cuda")
    shape = tb.rms_shape_of(x, dr, dy=dy)
    shape.eps = 1e-5
    tb.tri_rms_fwd(shape, x, dr, gamma, r, y, rstd)
    _check_forward(x, dr, gamma, 1e-5, tb.RmsOutput(y, rstd, r, None))
    ws = torch.empty(tb.tri_rms_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    tb.tri_rms_bwd(shape, r, gamma, rstd, dy, dr, dx, dgamma, ws)
    _check_backward(r, gamma, rstd, dy, dr, (dx, dgamma))
    for w in wide:
        assert (w[:off] == 7).all() and (w[off + M * C:] == 7).all()


def test_zeros_infinities_and_nans():
    """Each row answers for itself; a group that holds an infinity or a NaN is NaN in 8 bits; a row of zeros is zeros."""
    x = _normal((6, 300), torch.float32, 30)
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, 290] = float("inf")
    x[4] *= 1e-30
    got = tb.rms_forward(x, eight_bits=True)
    clean = [0, 5]
    _check_forward(x[clean], None, None, 1e-5, tb.RmsOutput(got.y[clean], got.rstd[clean], None, tb.Checkpoint(got.y8.q8[clean], got.y8.scale[clean])))
    assert (got.y[1] == 0).all() and (got.y8.q8[1] == 0).all() and (got.y8.scale[1] == 0).all()
    assert got.y[2].isnan().all() and tb.checkpoint_unpack(got.y8, torch.float32)[2].isnan().all()
    # (rstd is 0: finite values come to 0, the infinite one to NaN, and so does its group)
    assert (got.y[3, :256] == 0).all() and got.y[3, 290].isnan()
    assert (tb.checkpoint_unpack(got.y8, torch.float32)[3, :256] == 0).all() and tb.checkpoint_unpack(got.y8, torch.float32)[3, 256:].isnan().all()
    assert ((got.y[4].double() - x[4].double() * 1e-5 ** -0.5).abs() <= 4 * F * x[4].double().abs() * 1e-5 ** -0.5).all()


def test_tall():
    """More rows than one pass of the grid; 72 rows a lane group in the column sums."""
    x, res, dy = (_normal((700001, 128), torch.bfloat16, s) for s in (13, 14, 15))
    gamma = _normal((128,), torch.float32, 16, 0.3, 1.0)
    got = tb.rms_forward(x, gamma, res, eight_bits=True)
    _check_forward(x, res, gamma, 1e-5, got)
    _check_backward(got.r, gamma, got.rstd, dy, None, tb.rms_backward(got.r, gamma, got.rstd, dy))
