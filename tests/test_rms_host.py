"""Refusals of the RMS norm's calls (no GPU, nothing launched)."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def tb():
    from bwd_tri_attn_gb300 import _build, binding
    _build.build()
    binding.load()
    return binding


def shape(tb, M=4, C=64, dtype=0, eps=1e-5, ldx=0, ldres=0, lddy=0):
    return tb.RmsShape(M, ldx, ldres, lddy, C, dtype, eps)


FWD = ("x", "residual", "gamma", "r", "y", "rstd", "q8", "scale8")
BWD = ("r", "gamma", "rstd", "dy", "dr", "dx", "dgamma", "workspace")


def fwd(tb, s, nulls=(), **at):
    return tb.load().tri_rms_fwd(s, *[None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in FWD], None)


def bwd(tb, s, nulls=(), ws=1 << 40, **at):
    return tb.load().tri_rms_bwd(s, *[None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in BWD], ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("bad,code", [(dict(M=0), -1), (dict(C=0), -1), (dict(M=-3), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
                                      (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(ldx=63), -1),
                                      (dict(ldres=-64), -1), (dict(lddy=1), -1), (dict(C=8193), -2), (dict(M=1 << 41), -2),
                                      (dict(M=1 << 40, ldres=1 << 30), -2)])
def test_bad_shapes(tb, bad, code):
    s = shape(tb, **bad)
    assert fwd(tb, s) == code and bwd(tb, s) == code and tb.tri_rms_bwd_workspace_size(s) == 0


def test_pointers(tb):
    s = shape(tb)
    for nulls in (("x",), ("rstd",), ("residual",), ("r",), ("q8",), ("scale8",), ("y", "q8", "scale8")):
        assert fwd(tb, s, nulls) == -1
    for nulls in (("r",), ("rstd",), ("dy",), ("dx",)):
        assert bwd(tb, s, nulls) == -1
    for n in ("x", "residual", "r", "y", "gamma", "rstd", "scale8"):
        assert fwd(tb, s, **{n: FAKE + 1}) == -2
    for n in BWD:
        assert bwd(tb, s, **{n: FAKE + 1}) == -2
    need = tb.tri_rms_bwd_workspace_size(s)
    assert need >= 4 * 64 and bwd(tb, s, ws=need - 1) == -3 and bwd(tb, s, nulls=("workspace",)) == -3


def test_binding_refuses_before_the_library(tb):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.rms_forward(x)
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        tb.rms_forward(x.double())
    with pytest.raises(ValueError, match="at least one"):
        tb.rms_forward(x[:0])
    with pytest.raises(ValueError, match="residual .* must have x's shape"):
        tb.rms_forward(x, residual=x[:3])
    with pytest.raises(TypeError, match="residual must be"):
        tb.rms_forward(x, residual=x.float())
    with pytest.raises(TypeError, match="residual must be a torch.Tensor"):
        tb.rms_forward(x, residual=1.0)
    with pytest.raises(TypeError, match="gamma"):
        tb.rms_forward(x, x[0])
    with pytest.raises(ValueError, match="gamma"):
        tb.rms_forward(x, torch.zeros(63))
    with pytest.raises(ValueError, match="eight_bits"):
        tb.rms_forward(x, eight_bits="also")
    with pytest.raises(ValueError, match="evenly spaced"):
        tb.rms_forward(x, residual=x[:1].expand(4, 64))
    rstd = torch.zeros(4)
    with pytest.raises(ValueError, match="dy"):
        tb.rms_backward(x, None, rstd, x[:3])
    with pytest.raises(TypeError, match="dy must be"):
        tb.rms_backward(x, None, rstd, x.float())
    with pytest.raises(ValueError, match="rstd has"):
        tb.rms_backward(x, None, rstd[:3], x)
    with pytest.raises(ValueError, match="channels"):
        tb.rms_forward(torch.empty((1, 2 ** 32 + 8), dtype=torch.bfloat16, device="meta"))
