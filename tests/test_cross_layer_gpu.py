"""LayerNorm, its 8-bit checkpoint and cross attention together, as a layer of a decoder uses them: the
layer's gradients against the same formulas in 64 bits, a training step and a serving step captured into a
graph, and the layer around the triangle-attention block.

Tolerance of the gradients, in the norm of each tensor: the longest path from the loss to a gradient
passes sixteen roundings to BF16 (the normalised rows, q or k and v, P, O, the output projection, the
residual sum; on the way back the gradients of each, dS, and the output), of at most U = 2^-8 of the value
each; the checkpoint's steps are at most 1 / 254 of a group's largest magnitude, another 2^-8 or so
of the row's norm. Products with random matrices keep relative errors in the norm. 18 U in all.
"""
import pytest
import torch

from bwd_tri_attn_gb300 import autograd as ag
from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def parameters(c, cs, H, Hk, d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    p = {"g": 1.0 + normal(c, scale=0.2), "b": normal(c, scale=0.2), "gs": 1.0 + normal(cs, scale=0.2),
         "bs": normal(cs, scale=0.2), "wq": normal(H * d, c, scale=c ** -0.5).bfloat16(),
         "wkv": normal(2 * Hk * d, cs, scale=cs ** -0.5).bfloat16(), "wo": normal(c, H * d, scale=(H * d) ** -0.5).bfloat16()}
    return p, normal


def layer(p, x, states, lens, H, Hk, d, checkpoint=False):
    B, T, S = x.shape[0], x.shape[1], states.shape[1]
    q = torch.nn.functional.linear(ag.layer_norm(x, p["g"], p["b"], checkpoint=checkpoint), p["wq"]).view(B, T, H, d)
    kv = torch.nn.functional.linear(ag.layer_norm(states, p["gs"], p["bs"], checkpoint=checkpoint), p["wkv"])
    kv = kv.view(B, S, 2, Hk, d)
    o = ag.cross_attention(q, kv[:, :, 0], kv[:, :, 1], kv_lens=lens)
    return x + torch.nn.functional.linear(o.flatten(2), p["wo"])


def layer64(p, x, states, lens, H, Hk, d):
    def norm(t, g, b):
        return (t - t.mean(-1, keepdim=True)) / torch.sqrt(t.var(-1, unbiased=False, keepdim=True) + 1e-5) * g + b

    B, T, S = x.shape[0], x.shape[1], states.shape[1]
    q = (norm(x, p["g"], p["b"]) @ p["wq"].T).view(B, T, H, d).transpose(1, 2)
    kv = (norm(states, p["gs"], p["bs"]) @ p["wkv"].T).view(B, S, 2, Hk, d)
    k, v = (kv[:, :, i].transpose(1, 2).repeat_interleave(H // Hk, 1) for i in (0, 1))
    dead = (torch.arange(S, device="cuda") >= lens[:, None])[:, None, None]
    s = (q @ k.transpose(2, 3) * d ** -0.5).masked_fill(dead, -torch.inf)
    o = torch.softmax(s, -1).nan_to_num(0.0) @ v  # (a sequence without states: zeros)
    return x + o.transpose(1, 2).flatten(2) @ p["wo"].T


def leaves(p, *inputs):
    """Fresh leaves, so that no other graph of theirs lives."""
    p = {n: t.detach().clone().requires_grad_() for n, t in p.items()}
    return p, [t.detach().clone().requires_grad_() for t in inputs]


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("B,T,S,c,cs,H,Hk,d,lens", [(2, 100, 333, 256, 384, 8, 2, 32, [333, 130]), (1, 1, 77, 128, 200, 4, 4, 64, [77]),
                                                    (2, 257, 128, 384, 128, 4, 1, 128, [0, 128])])
def test_gradients_of_a_layer(B, T, S, c, cs, H, Hk, d, lens, checkpoint):
    p, normal = parameters(c, cs, H, Hk, d)
    x, states, dout = normal(B, T, c).bfloat16(), normal(B, S, cs).bfloat16(), normal(B, T, c).bfloat16()
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, (a, s) = leaves(p, x, states)
    out = layer(q, a, s, lens, H, Hk, d, checkpoint)
    out.backward(dout)
    q64, (a64, s64) = leaves({n: t.double() for n, t in p.items()}, x.double(), states.double())
    want = layer64(q64, a64, s64, lens, H, Hk, d)
    want.backward(dout.double())
    assert tb.tri_attn_device_status() == 0
    pairs = {"out": (out, want), "x": (a.grad, a64.grad), "states": (s.grad, s64.grad),
             **{n: (q[n].grad, q64[n].grad) for n in p}}
    for n, (got, w) in pairs.items():
        assert got.isfinite().all(), n
        assert (got.double() - w).norm() <= 18 * U * w.norm(), n
    # the residual x and its gradient are most of "x": what the layer adds to them, too
    assert ((a.grad - dout).double() - (a64.grad - dout.double())).norm() <= 18 * U * (a64.grad - dout.double()).norm() + U * dout.double().norm()


def test_training_step_in_a_graph():
    B, T, S, c, cs, H, Hk, d = 2, 130, 300, 128, 192, 4, 2, 64
    p, normal = parameters(c, cs, H, Hk, d)
    data = [(normal(B, T, c).bfloat16(), normal(B, S, cs).bfloat16(), normal(B, T, c).bfloat16(),
             torch.tensor(n, dtype=torch.int32, device="cuda")) for n in ([300, 17], [0, 257])]

    def step(x, states, dout, lens):
        q, (a, s) = leaves(p, x, states)
        out = layer(q, a, s, lens, H, Hk, d, checkpoint=True)
        return [out.detach(), *torch.autograd.grad(out, [a, s, *q.values()], dout)]

    want = [step(*batch) for batch in data]
    static = [t.clone() for t in data[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static)
    for batch, results in zip(data, want):
        for t, n in zip(static, batch):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, results):
            assert torch.equal(g, w)
    assert tb.tri_attn_device_status() == 0


def test_serving_step_in_a_graph():
    """One token of each sequence at a time; the sequences' lengths change between replays."""
    B, S, c, H, Hk, d = 3, 1000, 256, 8, 2, 64
    p, normal = parameters(c, c, H, Hk, d)
    x = normal(B, 1, c).bfloat16()
    kv = normal(B, S, 2, Hk, d).bfloat16()
    lens = torch.tensor([S, 1, 130], dtype=torch.int32, device="cuda")

    def step():
        y = tb.norm_forward(x, p["g"], p["b"])[0]
        q = torch.nn.functional.linear(y, p["wq"]).view(B, 1, H, d)
        return tb.cross_forward(q, kv[:, :, 0], kv[:, :, 1], kv_lens=lens)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in ([S, 1, 130], [0, S, 511], [7, 0, 0]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        x.copy_(normal(B, 1, c))
        graph.replay()
        for g, w in zip(got, step()):
            assert torch.equal(g, w)
    assert tb.tri_attn_device_status() == 0


def test_layer_behind_the_triangle_attention_block():
    """Single tokens attend to a pair representation's rows, both blocks with 8-bit checkpoints."""
    N, c, H, d = 48, 128, 4, 32
    p, normal = parameters(c, c, H, H, d)
    block = ag.TriangleAttentionBlock(c, H, d, device="cuda", checkpoint=True)
    z = normal(1, N, N, c).bfloat16().requires_grad_()
    x = normal(1, N, c).bfloat16().requires_grad_()
    lens = torch.tensor([N * N], dtype=torch.int32, device="cuda")
    out = layer(p, x, (z + block(z)).view(1, N * N, c), lens, H, H, d, checkpoint=True)
    out.backward(normal(1, N, c).bfloat16())
    for t in (x, z, *block.parameters()):
        assert t.grad.isfinite().all() and t.grad.abs().max() > 0
    assert tb.tri_attn_device_status() == 0


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_another_stream(handle):
    """A call's results and workspace may be dropped while the stream that it was given has not begun it."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((2, n, 4, 64), generator=gen, device="cuda").bfloat16() for n in (300, 600, 600, 300))
    x, g = torch.randn((600, 256), generator=gen, device="cuda"), torch.ones(256, device="cuda")
    O, LSE = tb.cross_forward(q, k, v)
    y, mean, rstd = tb.norm_forward(x, g, g)
    kept = tb.checkpoint_pack(x)
    calls = [lambda s: tb.cross_forward(q, k, v, stream=s), lambda s: tb.cross_backward(q, k, v, O, LSE, do, stream=s),
             lambda s: tb.norm_forward(x, g, g, checkpoint=True, stream=s)[:3], lambda s: tb.norm_backward(x, g, mean, rstd, y, stream=s),
             lambda s: tb.checkpoint_pack(x, stream=s), lambda s: (tb.checkpoint_unpack(kept, torch.float32, stream=s),)]
    for call in calls:
        want = [t.clone() for t in call(None)]
        sizes = [t.numel() * t.element_size() for t in want] + [tb.tri_cross_bwd_workspace_size(tb.cross_shape_of(q, k, v))]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # (about 10 ms)
        call(stream)  # (the results are dropped at once)
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        got = call(stream)
        torch.cuda.synchronize()
        assert all((o == 7).all() for o in others)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tb.tri_attn_device_status() == 0
