"""Clipping of gradients whose axes lie in another order (of parameters kept transposed or channels-last). Tolerances as
in test_clip_gpu.py."""
import pytest
import torch

from bwd_tri_attn_gb300 import autograd, binding as tb
from tests.test_clip_gpu import DTYPES, T, check, norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("share", [0.5, 2.0])
def test_permuted_gradients(dtype, share):
    gen = torch.Generator(device="cuda").manual_seed(1)
    t = torch.randn(6, 7, 30, 41, generator=gen, device="cuda").to(dtype)
    grads = [t[0, 0].clone().t(), t.clone().permute(3, 1, 0, 2), t.clone(memory_format=torch.channels_last), t[1].clone()]
    before = [g.clone() for g in grads]
    most = share * norm64(before)
    out = [torch.full_like(g, 3) for g in grads]
    assert all(o.stride() == g.stride() for o, g in zip(out, grads))
    check(grads, before, most, tb.clip_gradients(grads, most, out=out), out)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    check(grads, before, most, tb.clip_gradients(grads, most), grads)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))


def test_parameters_kept_transposed():
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.nn.Parameter(torch.randn(64, 96, generator=gen, device="cuda").t())
    c = torch.nn.Conv2d(8, 16, 3, device="cuda").to(memory_format=torch.channels_last)
    x = torch.randn(5, 96, generator=gen, device="cuda")
    (x @ w).square().sum().backward()
    c.weight.grad = torch.randn(c.weight.shape, generator=gen, device="cuda").to(memory_format=torch.channels_last)
    assert not w.grad.is_contiguous() and not c.weight.grad.is_contiguous()
    grads = [w.grad, c.weight.grad]
    before = [g.clone() for g in grads]
    want = norm64(before)
    norm = autograd.clip_grad_norm_([w, *c.parameters()], 0.25 * want)
    check(grads, before, 0.25 * want, norm, grads)
    assert abs(norm.item() - want) <= T * want
