"""Gradients that share memory: the norm reads them, as often as they are named; what clipping writes lies apart.
Tolerances as in test_clip_gpu.py."""
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


def test_clipping_refuses_tensors_that_share_memory():
    flat = gradients([4000], dtypes=[torch.float32])[0]
    g, h = flat[:1500], flat[2000:3500]
    before, other = flat.clone(), torch.empty_like(flat)
    for grads, out in (([g, h], [h, g]), ([g, flat[1499:3000]], None), ([g, h], [other[:1500], other[1499:2999]]),
                       ([g], [flat[1:1501]]), ([g, h], [other[:1500], g])):
        with pytest.raises(ValueError, match="shares memory"):
            tb.clip_gradients(grads, 1.0, out=out)
    torch.cuda.synchronize()
    assert torch.equal(flat, before)
    most = 0.5 * norm64([g, h])
    tb.clip_gradients([g, h], most, out=[g, other[:1500]])  # (one in place, one apart)
    by = most / (2 * most + 1e-6)
    assert torch.allclose(g, before[:1500] * by, rtol=4 * T, atol=0) and torch.allclose(other[:1500], before[2000:3500] * by, rtol=4 * T, atol=0)
    assert torch.equal(flat[1500:], before[1500:])
