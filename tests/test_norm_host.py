"""Refusals of the LayerNorm and checkpoint calls (no GPU, nothing launched)."""
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


def _shape(tb, M=4, C=64, dtype=0, eps=1e-5, ldx=0, lddy=0):
    return tb.NormShape(M, ldx, lddy, C, dtype, eps)


BAD_SHAPES = [(dict(M=0), -1), (dict(C=0), -1), (dict(M=-3), -1), (dict(C=-1), -1), (dict(dtype=3), -1),
              (dict(dtype=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
              (dict(ldx=63), -1), (dict(lddy=-64), -1), (dict(M=1 << 41), -2), (dict(M=1 << 40, ldx=1 << 30), -2)]


def _call(fn, shape, names, nulls=(), **at):
    args = [None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in names]
    return args


FWD = ("x", "gamma", "beta", "y", "mean", "rstd", "q8", "scale8")
BWD = ("x", "q8", "scale8", "gamma", "mean", "rstd", "dy", "dx", "dgamma", "dbeta", "workspace")


def fwd(tb, shape, nulls=(), **at):
    return tb.load().tri_norm_fwd(shape, *_call("fwd", shape, FWD, nulls, **at), None)


def bwd(tb, shape, nulls=("q8", "scale8"), ws=1 << 30, **at):
    return tb.load().tri_norm_bwd(shape, *_call("bwd", shape, BWD, nulls, **at), ctypes.c_size_t(ws), None)


def pack(tb, shape, nulls=(), **at):
    return tb.load().tri_ckpt_pack(shape, *_call("pack", shape, ("x", "q8", "scale8"), nulls, **at), None)


def unpack(tb, shape, nulls=(), **at):
    return tb.load().tri_ckpt_unpack(shape, *_call("unpack", shape, ("q8", "scale8", "x"), nulls, **at), None)


@pytest.mark.parametrize("bad,code", BAD_SHAPES)
def test_bad_shapes(tb, bad, code):
    s = _shape(tb, **bad)
    for call in (fwd, bwd, pack, unpack):
        assert call(tb, s) == code
    assert tb.tri_norm_bwd_workspace_size(s) == 0


def test_too_wide(tb):
    s = _shape(tb, C=8193)
    assert fwd(tb, s) == -2 and bwd(tb, s) == -2 and tb.tri_norm_bwd_workspace_size(s) == 0


@pytest.mark.parametrize("null", ["x", "y", "mean", "rstd", "q8", "scale8"])
def test_forward_needs(tb, null):
    assert fwd(tb, _shape(tb), nulls=(null,)) == -1


@pytest.mark.parametrize("nulls", [("x", "q8", "scale8"), (), ("scale8",), ("q8", "scale8", "mean"), ("q8", "scale8", "rstd"),
                                   ("q8", "scale8", "dy"), ("q8", "scale8", "dx"), ("q8", "scale8", "dgamma"),
                                   ("q8", "scale8", "dbeta"), ("x", "q8"), ("x", "scale8")])
def test_backward_needs(tb, nulls):
    assert bwd(tb, _shape(tb), nulls=nulls) == -1


def test_backward_workspace(tb):
    s = _shape(tb, M=1000, C=256)
    need = tb.tri_norm_bwd_workspace_size(s)
    assert need >= 2 * 4 * 256
    assert bwd(tb, s, ws=need - 1) == -3
    assert bwd(tb, s, nulls=("q8", "scale8", "workspace")) == -3


@pytest.mark.parametrize("name,off", [("x", 1), ("y", 1), ("gamma", 2), ("beta", 1), ("mean", 2), ("rstd", 2), ("scale8", 2)])
def test_forward_alignment(tb, name, off):
    assert fwd(tb, _shape(tb), **{name: FAKE + off}) == -2


@pytest.mark.parametrize("name", ["x", "dy", "dx", "gamma", "mean", "rstd", "dgamma", "dbeta", "workspace"])
def test_backward_alignment(tb, name):
    assert bwd(tb, _shape(tb), **{name: FAKE + 1}) == -2


@pytest.mark.parametrize("null", ["x", "q8", "scale8"])
def test_checkpoint_needs(tb, null):
    assert pack(tb, _shape(tb), nulls=(null,)) == -1
    assert unpack(tb, _shape(tb), nulls=(null,)) == -1


def test_checkpoint_alignment(tb):
    for call in (pack, unpack):
        assert call(tb, _shape(tb), x=FAKE + 1) == -2
        assert call(tb, _shape(tb), scale8=FAKE + 2) == -2
    assert pack(tb, _shape(tb, dtype=2), x=FAKE + 2) == -2


def test_binding_refuses_before_the_library(tb):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.norm_forward(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.checkpoint_pack(x)
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        tb.norm_forward(x.double())
    with pytest.raises(TypeError, match="Tensor"):
        tb.norm_forward([1.0])
    with pytest.raises(ValueError, match="at least one"):
        tb.norm_forward(x[:0])
    with pytest.raises(ValueError, match="at least one"):
        tb.norm_forward(x[:, :0])
    with pytest.raises(ValueError, match="evenly spaced"):
        tb.norm_forward(x.t())
    with pytest.raises(ValueError, match="evenly spaced"):
        tb.norm_forward(x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="evenly spaced"):
        tb.norm_forward(torch.zeros(3, 4, 64)[:, :2, :8])
    with pytest.raises(TypeError, match="gamma"):
        tb.norm_forward(x, x[0])
    with pytest.raises(ValueError, match="gamma"):
        tb.norm_forward(x, torch.zeros(63))
    mean = torch.zeros(4)
    with pytest.raises(ValueError, match="shape"):
        tb.norm_backward(x, None, mean, mean, x[:3])
    with pytest.raises(TypeError, match="x must be"):
        tb.norm_backward(x.float(), None, mean, mean, x)
    with pytest.raises(ValueError, match="mean has"):
        tb.norm_backward(x, None, mean[:3], mean, x)
    with pytest.raises(ValueError, match="scale has"):
        tb.norm_backward(tb.Checkpoint(x.to(torch.int8), torch.zeros(3, 1)), None, mean, mean, x)
    with pytest.raises(TypeError, match="q8"):
        tb.checkpoint_unpack((x, torch.zeros(4, 1)))
    with pytest.raises(TypeError, match="x must be"):
        tb.checkpoint_unpack((x.to(torch.int8), torch.zeros(4, 1)), dtype=torch.float64)


def test_row_strides(tb):
    x = torch.zeros(3, 5, 32)
    assert tb.norm_shape_of(x).ldx == 32 and tb.norm_shape_of(x[..., :7]).ldx == 32
    assert tb.norm_shape_of(x[0, :, 3:9]).ldx == 32 and tb.norm_shape_of(x[1:2, 2:3, :4]).M == 1
    assert tb.norm_shape_of(x[:, 0, :4]).ldx == 160
    assert tb.norm_shape_of(x[0, 0]).M == 1
