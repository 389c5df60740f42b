"""Refusals of the cross-attention calls (no GPU, nothing launched)."""
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


FWD = ("Q", "K", "V", "mask", "kv_lens", "O", "LSE", "workspace")
BWD = ("Q", "K", "V", "mask", "kv_lens", "O", "LSE", "dO", "dQ", "dK", "dV", "workspace")


def shape(tb, B=2, T=30, S=200, H=4, Hk=2, d=64, scale=0.125, q=None, k=None, v=None):
    three = ctypes.c_int64 * 3
    return tb.CrossShape(B, T, S, H, Hk, d, scale, three(*(q or (T * H * d, H * d, d))),
                         three(*(k or (S * Hk * d, Hk * d, d))), three(*(v or (S * Hk * d, Hk * d, d))))


def fwd(tb, s, nulls=(), ws=1 << 34, **at):
    args = [None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in FWD]
    return tb.load().tri_cross_fwd(s, *args, ctypes.c_size_t(ws), None)


def bwd(tb, s, nulls=(), ws=1 << 34, **at):
    args = [None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in BWD]
    return tb.load().tri_cross_bwd(s, *args, ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), -1), (dict(T=0), -1), (dict(S=0), -1), (dict(H=0), -1), (dict(Hk=0), -1), (dict(d=0), -1),
    (dict(B=-1), -1), (dict(H=5), -1), (dict(Hk=8), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(d=4), -2), (dict(d=12), -2), (dict(d=136), -2), (dict(B=65536), -2), (dict(H=2048), -2),
    (dict(T=(1 << 30) + 1), -2), (dict(S=(1 << 30) + 1), -2),
    (dict(S=(1 << 26) + 1), -2), (dict(T=(1 << 25) + 1), -2), (dict(H=1000, Hk=1, T=67109), -2), (dict(B=60000, T=1 << 29, S=1 << 29), -2),
    (dict(q=(7680, 260, 64)), -2), (dict(q=(7680, 256, 0)), -2), (dict(k=(0, 128, 64)), -2), (dict(v=(25600, -128, 64)), -2),
    (dict(k=(25600, 128, 60)), -2), (dict(v=(1 << 40, 128, 64)), -2)])
def test_bad_shapes(tb, bad, code):
    s = shape(tb, **bad)
    assert fwd(tb, s) == code and bwd(tb, s) == code
    assert tb.tri_cross_fwd_workspace_size(s) == 0 and tb.tri_cross_bwd_workspace_size(s) == 0


@pytest.mark.parametrize("null", ["Q", "K", "V", "O", "LSE"])
def test_forward_needs(tb, null):
    assert fwd(tb, shape(tb), nulls=(null,)) == -1


@pytest.mark.parametrize("null", ["Q", "K", "V", "O", "LSE", "dO", "dQ", "dK", "dV"])
def test_backward_needs(tb, null):
    assert bwd(tb, shape(tb), nulls=(null,)) == -1


@pytest.mark.parametrize("name", [n for n in BWD if n != "mask"])
def test_alignment(tb, name):
    off = 2 if name == "kv_lens" else 8
    assert bwd(tb, shape(tb), **{name: FAKE + off}) == -2
    if name in FWD:
        assert fwd(tb, shape(tb), **{name: FAKE + off}) == -2


def test_binding_refuses_before_the_library(tb):
    bf = torch.bfloat16
    q, k = torch.zeros(2, 30, 4, 64, dtype=bf), torch.zeros(2, 200, 2, 64, dtype=bf)
    with pytest.raises(TypeError, match="Q must be"):
        tb.cross_forward(q.float(), k, k)
    with pytest.raises(TypeError, match="Tensor"):
        tb.cross_forward(None, k, k)
    with pytest.raises(ValueError, match="four axes"):
        tb.cross_forward(q[0], k, k)
    with pytest.raises(ValueError, match="V has shape"):
        tb.cross_forward(q, k, k[:, :199])
    with pytest.raises(ValueError, match="K has shape"):
        tb.cross_forward(q, k[:1], k)
    with pytest.raises(ValueError, match="K has shape"):
        tb.cross_forward(q, k[..., :32], k)
    with pytest.raises(ValueError, match="last axis"):
        tb.cross_forward(q, k.transpose(1, 3).contiguous().transpose(1, 3), k)
    with pytest.raises(ValueError, match="mask has"):
        tb.cross_forward(q, k, k, torch.ones(2, 199, dtype=torch.bool))
    with pytest.raises(TypeError, match="mask must be"):
        tb.cross_forward(q, k, k, torch.ones(2, 200))
    with pytest.raises(ValueError, match="mask must be contiguous"):
        tb.cross_forward(q, k, k, torch.ones(200, 2, dtype=torch.bool).t())
    with pytest.raises(TypeError, match="kv_lens must be"):
        tb.cross_forward(q, k, k, None, torch.ones(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="kv_lens has"):
        tb.cross_forward(q, k, k, None, torch.ones(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.cross_forward(q, k, k)
    lse = torch.zeros(2, 4, 30)
    with pytest.raises(ValueError, match="dO has"):
        tb.cross_backward(q, k, k, q, lse, q[:1].contiguous())
    with pytest.raises(ValueError, match="LSE has"):
        tb.cross_backward(q, k, k, q, lse[:1], q)
    with pytest.raises(ValueError, match="dO must be contiguous"):
        tb.cross_backward(q, k, k, q, lse, torch.zeros(2, 4, 30, 64, dtype=bf).transpose(1, 2))


def test_what_autograd_copies():
    from bwd_tri_attn_gb300.autograd import _spaced
    kv = torch.zeros(2, 20, 2, 3, 16, dtype=torch.bfloat16)
    k = kv[:, :, 1]
    assert _spaced(k) is k                                   # part of a fused projection
    t = torch.zeros(2, 3, 20, 16, dtype=torch.bfloat16).transpose(1, 2)
    assert _spaced(t) is t                                   # heads before positions
    for bad in (torch.zeros(2, 20, 3, 20, dtype=torch.bfloat16)[..., 1:17],       # an unaligned start
                torch.zeros(2, 20, 3, 20, dtype=torch.bfloat16)[..., :16],        # strides of 20 elements
                torch.zeros(2, 20, 1, 16, dtype=torch.bfloat16).expand(2, 20, 3, 16),
                torch.zeros(2, 20, 16, 3, dtype=torch.bfloat16).transpose(2, 3)):
        c = _spaced(bad)
        assert c is not bad and c.is_contiguous() and torch.equal(c, bad) and c.data_ptr() % 16 == 0
