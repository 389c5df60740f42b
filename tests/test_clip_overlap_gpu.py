"""Gradients that share memory: the norm reads them, as often as they are named; what clipping writes lies apart.
Tolerances as in test_clip_gpu.py."""
import math

import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from tests.test_clip_gpu import DTYPES, T, gradients, norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_norm_of_tensors_that_share_memory(dtype):
    g, h = gradients([5000, 77], dtypes=[dtype])
    flat = gradients([3000], 1, dtypes=[dtype])[0]
    for grads in ([g, g], [g, h, g, h, g], [flat[:2000], flat[1000:], flat], [g[:0], g, g[:0]]):
        before = [t.clone() for t in grads]
        want = norm64(grads)
        assert abs(tb.gradient_norm(grads).item() - want) <= T * want
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
