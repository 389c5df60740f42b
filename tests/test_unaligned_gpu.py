"""Autograd with inputs and gradients that are contiguous but begin off the 16-byte boundaries (parts of a
concatenation): the same bits as with fresh tensors."""
import pytest
import torch

from bwd_tri_attn_gb300 import autograd as ag
from bwd_tri_attn_gb300 import binding as tb
from bwd_tri_attn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def off(t):
    """The same values, one element behind a boundary."""
    if t is None:
        return None
    part = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    part.copy_(t)
    assert part.is_contiguous() and part.data_ptr() % 16 != 0
    return part


def cases():
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    a = {n: t.cuda() for n, t in wl.make_inputs(B=1, S=24, N=72, H=2, d=32, seed=4, mask=("tail", 9)).items()}
    m = {n: t.cuda() for n, t in wl.make_module_inputs(1, 40, 128, 4, 32, seed=5, mask=("tail", 3)).items()}
    x, g, b = normal(50, 96), torch.rand(96, device="cuda") + 0.5, torch.rand(96, device="cuda")
    mask = torch.rand((2, 130), generator=gen, device="cuda") < 0.9
    lens = torch.tensor([130, 77], dtype=torch.int32, device="cuda")
    return {
        "cross_attention": (ag.cross_attention, [normal(2, 60, 4, 64), normal(2, 130, 2, 64), normal(2, 130, 2, 64)], [mask, lens]),
        "layer_norm": (ag.layer_norm, [x, g, b], []),
        "layer_norm_checkpoint": (lambda *t: ag.layer_norm(*t, checkpoint=True), [x, g, b], []),
        "triangle_attention": (ag.triangle_attention, [a[n] for n in ("Q", "K", "V", "bias")], [a["mask"]]),
        "triangle_multiplication": (ag.triangle_multiplication, [normal(1, 40, 40, 24) for _ in range(4)], []),
        "triangle_attention_block": (lambda *t: ag.triangle_attention_block(*t, 4, 32),
                                     [m[n] for n in ("z", "gamma", "beta", "W", "wb", "Wo")], [m["mask"]]),
    }


NAMES = ["cross_attention", "layer_norm", "layer_norm_checkpoint", "triangle_attention", "triangle_multiplication",
         "triangle_attention_block"]


@pytest.mark.parametrize("name", NAMES)
def test_inputs_and_gradients_off_the_boundaries(name):
    call, leaves, others = cases()[name]

    def run(place, dout=None):
        xs = [place(t).requires_grad_() for t in leaves]
        out = call(*xs, *[place(t) for t in others])
        if dout is None:
            dout = torch.randn(out.shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(out.dtype)
        return dout, [out.detach(), *torch.autograd.grad(out, xs, place(dout))]

    dout, want = run(torch.clone)
    _, got = run(off, dout)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tb.tri_attn_device_status() == 0


def test_gradient_of_a_concatenation():
    """A scalar before O in one flat tensor: O's gradient is the concatenation's from its second element on."""
    _, (q, k, v), _ = cases()["cross_attention"]
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    dO = torch.randn(q.shape, device="cuda").bfloat16()
    want = torch.autograd.grad(ag.cross_attention(q, k, v), (q, k, v), dO)
    flat = torch.cat([torch.ones(1, dtype=torch.bfloat16, device="cuda"), ag.cross_attention(q, k, v).flatten()])
    got = torch.autograd.grad(flat, (q, k, v), torch.cat([torch.ones(1, dtype=torch.bfloat16, device="cuda"), dO.flatten()]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
