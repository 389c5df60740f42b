"""The gradients' norm and clipping (include/tri_clip.h) against the formula in 64 bits.

Tolerances: 16 squares are added in FP32 (under 2^-20 of their sum), the rest in FP64, then one rounding: the norm is within
2^-21 (half of that, for the root) + 2^-24 of the 64-bit one, T = 2^-20 bounds it. The factor adds a sum and a quotient
(2 x 2^-24): 2 T, and an output half a step of its type (torch.finfo(t).eps / 2, or of its smallest number) more.
"""
import math

import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

T = 2.0 ** -20
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def gradients(sizes, seed=0, scale=0.1, dtypes=DTYPES):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(math.fsum(g.double().square().sum().item() for g in grads))


def check(grads, before, most, norm, out):
    want = norm64(before)
    assert abs(norm.item() - want) <= T * want
    by = min(1.0, most / (want + 1e-6))
    for o, g in zip(out, before):
        assert o.dtype == g.dtype and o.shape == g.shape
        tol = (torch.finfo(g.dtype).eps / 2 + 2 * T) * by * g.double().abs() + torch.finfo(g.dtype).smallest_normal * torch.finfo(g.dtype).eps
        assert ((o.double() - by * g.double()).abs() <= tol).all()


SIZES = [[1], [7, 0, 1], [4096], [4095, 4097, 3], [100000, 5, 33333], [1] * 95, [3] * 96, [2] * 97, [1000] * 300, [5000000, 17, 300]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("share", [0.25, 4.0])
def test_in_place_and_into_others(sizes, share):
    grads = gradients(sizes)
    before = [g.clone() for g in grads]
    most = share * norm64(before)
    out = [torch.full_like(g, 7) for g in grads]
    assert torch.equal(tb.gradient_norm(grads), tb.clip_gradients(grads, most, out=out))
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    check(grads, before, most, tb.gradient_norm(grads), out)
    norm = tb.clip_gradients(grads, most)
    check(grads, before, most, norm, grads)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 1), (0, 5), (7, 0)])
def test_tensors_that_start_anywhere(dtype, a, b):
    """Nothing beside a tensor is read (it is NaN) or written."""
    for n in (1, 5, 8, 4096, 20001):
        wide, other = (torch.full((n + 32,), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        g, o = wide[8 + a:8 + a + n], other[8 + b:8 + b + n]
        g.copy_(gradients([n], n)[0])
        before = g.clone()
        most = 0.5 * norm64([before])
        check([g], [before], most, tb.clip_gradients([g], most, out=[o]), [o])
        check([g], [before], most, tb.clip_gradients([g], most), [g])
        for w, p in ((wide, a), (other, b)):
            assert w[:8 + p].isnan().all() and w[8 + p + n:].isnan().all()


@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-12, 1e12, 1e25, 1e36])
def test_range(scale):
    """Squares that FP32 cannot hold."""
    g = gradients([3000, 40001], 1, 1.0, [torch.float32])
    for t in g:
        t.mul_(scale)
    want = norm64(g)
    norm = tb.gradient_norm(g).item()
    assert abs(norm - want) <= T * want
    mixed = g + gradients([500], 2, 1.0, [torch.float32])
    assert abs(tb.gradient_norm(mixed).item() - norm64(mixed)) <= T * norm64(mixed)


def test_zeros_infinities_and_nans():
    g = gradients([1000, 50], 3, dtypes=[torch.float32])
    for t in g:
        t.zero_()
    assert tb.clip_gradients(g, 1.0).item() == 0.0 and all((t == 0).all() for t in g)
    g = gradients([1000, 50], 3, dtypes=[torch.float32])
    g[1][3] = float("inf")
    assert tb.clip_gradients(g, 1.0).item() == math.inf
    assert (g[0] == 0).all() and g[1][3].isnan()
    g = gradients([1000, 50], 3, dtypes=[torch.float32])
    g[0][999] = float("nan")
    assert math.isnan(tb.clip_gradients(g, 1.0).item()) and all(t.isnan().all() for t in g)
    g = gradients([1000, 50], 3)
    before = [t.clone() for t in g]
    assert tb.clip_gradients(g, math.inf).item() == tb.gradient_norm(before).item()
    assert all(torch.equal(a, b) for a, b in zip(g, before))
    tb.clip_gradients(g, 0.0)
    assert all((t == 0).all() for t in g)
    assert tb.clip_gradients([], 1.0).item() == 0.0 and tb.gradient_norm([]).item() == 0.0


def test_captured():
    """A captured call reads the gradients as they are at each replay."""
    grads = gradients([3000, 129, 70000])
    out = [torch.empty_like(g) for g in grads]
    tb.clip_gradients(grads, 1.0, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = tb.clip_gradients(grads, 1.0, out=out)
    for seed in (5, 6):
        for g, n in zip(grads, gradients([3000, 129, 70000], seed, 0.01 * seed)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        check(grads, grads, 1.0, norm, out)
