"""Sizes that do not fit the C structures' 32-bit fields are refused before they are cut (no GPU; the tensors are
meta tensors, without memory)."""
import ctypes

import pytest
import torch

from bwd_tri_attn_gb300 import _build, binding as tb

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    tb.load()


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("C", [2 ** 31 - 127, 2 ** 31, 2 ** 32 + 8, 2 ** 33])
def test_channels(C):
    x = meta(1, C)
    for call in (lambda: tb.checkpoint_pack(x), lambda: tb.norm_forward(x), lambda: tb.norm_forward(x, checkpoint=True),
                 lambda: tb.norm_backward(x, None, meta(1, dtype=torch.float32), meta(1, dtype=torch.float32), x),
                 lambda: tb.checkpoint_unpack((meta(1, C, dtype=torch.int8), meta(1, (C + 127) // 128, dtype=torch.float32)))):
        with pytest.raises(ValueError, match="channels"):
            call()
    assert tb.norm_shape_of(meta(1, 2 ** 31 - 128)).C == 2 ** 31 - 128


@pytest.mark.parametrize("C", [2 ** 31 - 127, 2 ** 31 - 1])
def test_channels_of_the_c_calls(C):
    shape = tb.NormShape(1, 0, 0, C, 0, 1e-5)
    three = [ctypes.c_void_p(FAKE)] * 3
    assert tb.load().tri_ckpt_pack(shape, *three, None) == -2
    assert tb.load().tri_ckpt_unpack(shape, *three, None) == -2


@pytest.mark.parametrize("q,k", [((1, 2, 4, 64), (1, 2 ** 32 + 8, 2, 64)), ((1, 2 ** 32 + 1, 4, 64), (1, 5, 2, 64)),
                                 ((2 ** 32 + 1, 1, 1, 8), (2 ** 32 + 1, 1, 1, 8)), ((1, 2, 2 ** 32 + 4, 64), (1, 5, 2, 64)),
                                 ((1, 2, 4, 64), (1, 5, 2 ** 31, 64)), ((1, 2, 4, 2 ** 32 + 64), (1, 5, 2, 2 ** 32 + 64))])
def test_axes_of_cross_attention(q, k):
    Q, K = meta(*q), meta(*k)
    lse = meta(q[0], q[2], q[1], dtype=torch.float32)
    for call in (lambda: tb.cross_shape_of(Q, K, K), lambda: tb.cross_forward(Q, K, K),
                 lambda: tb.cross_backward(Q, K, K, Q, lse, Q)):
        with pytest.raises(ValueError, match="too long"):
            call()
