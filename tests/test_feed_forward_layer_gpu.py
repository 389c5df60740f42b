"""The relative position bias, RMS norm, gated feed-forward block and clipping together, as a trunk's training step uses them
around the triangle attention: gradients against the same formulas in 64 bits, the step captured into a graph, masters and
what is frozen, calls on other streams and from fresh threads.

Tolerance of the gradients, in the norm of each tensor: the longest path from the loss to a gradient passes 20 roundings
to BF16 (bias, q, k, v, P, O, the projection, the sum, y, a or u, h, out; on the way back the gradients of each), of at most
U = 2^-8 of the value each; the 8-bit checkpoint's steps are at most 1 / 254 of a group's largest magnitude, another 2^-8 or
so of the row's norm. Products with random matrices keep relative errors in the norm. 22 U in all.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

from bwd_tri_attn_gb300 import autograd as ag
from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
STARTS = tb.relpos_starts(16, 24)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def parameters(C, F, H, d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return gen, {"table": normal(gen, 2 * len(STARTS), H), "wqkv": normal(gen, 3 * H * d, C, std=C ** -0.5).bfloat16().float(),
                 "wo": normal(gen, C, H * d, std=(H * d) ** -0.5).bfloat16().float(), "gamma": 1 + normal(gen, C, std=0.2),
                 "wg": normal(gen, F, C, std=C ** -0.5).bfloat16().float(), "wu": normal(gen, F, C, std=C ** -0.5).bfloat16().float(),
                 "wd": normal(gen, C, F, std=F ** -0.5).bfloat16().float()}


def step(p, z, base, H, d, act, checkpoint=False, fused=True):
    """A row attention with the relative position's bias, then the feed-forward layer, on z [B, N, N, C]."""
    B, N, _, C = z.shape
    bias = ag.relative_position_bias(p["table"], STARTS, N, B=B, base=base)
    q, k, v = (torch.nn.functional.linear(z, p["wqkv"].bfloat16()).view(B, N, N, 3, H, d)[:, :, :, i] for i in range(3))
    o = ag.triangle_attention(q, k, v, bias).flatten(3)
    o = torch.nn.functional.linear(o, p["wo"].bfloat16())
    if fused:
        out, r = ag.feed_forward_layer(o, z, p["gamma"], p["wg"], p["wu"], p["wd"], act, checkpoint=checkpoint)
    else:
        y, r = ag.rms_norm(o, p["gamma"], z)
        out = ag.gated_feed_forward(y, p["wg"], p["wu"], p["wd"], act, checkpoint=checkpoint)
    return r + out


def step64(p, z, base, H, d, act):
    B, N, _, C = z.shape
    i = torch.arange(N, device="cuda")
    far = i[None, :] - i[:, None]
    rows = torch.searchsorted(torch.tensor(STARTS, device="cuda"), far.abs(), right=True) - 1 + len(STARTS) * (far > 0)
    bias = base + p["table"][rows].permute(2, 0, 1)
    q, k, v = ((z @ p["wqkv"].T).view(B, N, N, 3, H, d)[:, :, :, j].transpose(2, 3) for j in range(3))
    s = q @ k.transpose(3, 4) * d ** -0.5 + bias[:, None]
    o = (torch.softmax(s, -1) @ v).transpose(2, 3).flatten(3) @ p["wo"].T
    r = o + z
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-5) * p["gamma"]
    a, u = y @ p["wg"].T, y @ p["wu"].T
    f = torch.nn.functional.silu(a) if act == "silu" else torch.nn.functional.gelu(a) if act == "gelu" else torch.sigmoid(a)
    return r + (f * u) @ p["wd"].T


def leaves(p, *inputs):
    """Fresh leaves, so that no other graph of theirs lives."""
    return {n: t.detach().clone().requires_grad_() for n, t in p.items()}, [t.detach().clone().requires_grad_() for t in inputs]


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("B,N,C,F,H,d,act", [(1, 40, 128, 256, 4, 32, "silu"), (2, 33, 72, 200, 2, 16, "gelu"), (1, 160, 64, 128, 2, 16, "sigmoid")])
def test_gradients_of_a_step(B, N, C, F, H, d, act, fused, checkpoint):
    gen, p = parameters(C, F, H, d)
    z, base, dout = normal(gen, B, N, N, C).bfloat16(), normal(gen, B, H, N, N).bfloat16(), normal(gen, B, N, N, C).bfloat16()
    q, (zz, bb) = leaves(p, z, base)
    out = step(q, zz, bb, H, d, act, checkpoint, fused)
    out.backward(dout)
    q64, (z64, b64) = leaves({n: t.double() for n, t in p.items()}, z.double(), base.double())
    want = step64(q64, z64, b64, H, d, act)
    want.backward(dout.double())
    assert tb.tri_attn_device_status() == 0
    for n, got, w in [("out", out, want), ("z", zz.grad, z64.grad), ("base", bb.grad, b64.grad), *((n, q[n].grad, q64[n].grad) for n in p)]:
        assert got.isfinite().all(), n
        assert (got.double() - w).norm() <= 22 * U * w.norm(), n
    before = [t.grad.clone() for t in q.values()]
    size = math.sqrt(sum(g.double().square().sum().item() for g in before))
    norm = ag.clip_grad_norm_(q.values(), 0.5 * size)
    assert abs(norm.item() - size) <= 2.0 ** -20 * size
    for t, g in zip(q.values(), before):
        assert ((t.grad - 0.5 * g).abs() <= 2.0 ** -19 * g.abs()).all()


def test_clipping_shows_as_a_write():
    """What autograd keeps of a gradient may not be read after it was clipped in place."""
    w = torch.ones(40, device="cuda", requires_grad=True)
    other = torch.ones(40, device="cuda", requires_grad=True)
    w.grad = torch.full((40,), 3.0, device="cuda")
    y = other * w.grad
    ag.clip_grad_norm_([w, other], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_step_in_a_graph():
    """Forward, backward and clipping captured, replayed on other data."""
    B, N, C, F, H, d = 1, 36, 64, 192, 2, 32
    gen, p = parameters(C, F, H, d)
    data = [(normal(gen, B, N, N, C).bfloat16(), normal(gen, B, H, N, N).bfloat16(), normal(gen, B, N, N, C).bfloat16()) for _ in range(3)]

    def once(z, base, dout):
        q, (zz, bb) = leaves(p, z, base)
        out = step(q, zz, bb, H, d, "silu", checkpoint=True)
        grads = torch.autograd.grad(out, [zz, bb, *q.values()], dout)
        norm = tb.clip_gradients(list(grads[2:]), 1.0)
        return [out.detach(), norm, *grads]

    want = [once(*batch) for batch in data]
    static = [t.clone() for t in data[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once(*static)
    for batch, results in zip(data, want):
        for t, n in zip(static, batch):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, results))
    assert tb.tri_attn_device_status() == 0


@pytest.mark.parametrize("checkpoint", [False, True])
def test_module_with_masters(checkpoint):
    """FP32 masters get FP32 gradients, more exact than BF16 ones; without gradients nothing is kept."""
    torch.manual_seed(1)
    layer = ag.FeedForwardLayer(C=136, F=264, act="gelu", device="cuda", checkpoint=checkpoint)
    x, res, dout = (torch.randn(5, 60, 136, device="cuda").bfloat16() for _ in range(3))
    out, r = layer(x, res)
    assert torch.equal(r, x + res)
    out.backward(dout)
    with torch.no_grad():
        again, _ = layer(x, res)
    if not checkpoint:
        bf = [getattr(layer, n).detach().bfloat16() for n in ("Wg", "Wu", "Wd")]
        got = tb.rms_forward(x, layer.gamma.detach(), res)
        o, a, u = tb.ffn_forward(got.y, *bf, act="gelu", keep=True)
        exact = tb.ffn_backward(got.y, *bf, a, u, dout, act="gelu", weight_dtype=torch.float32)
        rounded = tb.ffn_backward(got.y, *bf, a, u, dout, act="gelu")
        assert torch.equal(out, again) and torch.equal(out, o)
        for n, e, b in zip(("Wg", "Wu", "Wd"), exact[1:], rounded[1:]):
            assert torch.equal(getattr(layer, n).grad, e) and torch.equal(e.bfloat16(), b)
    assert all(t.grad.dtype == torch.float32 and t.grad.abs().max() > 0 for t in layer.parameters())


def test_what_is_frozen():
    """Frozen weights or inputs: the other gradients stay the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, dout = normal(gen, 70, 64).bfloat16(), normal(gen, 70, 64).bfloat16()
    w = [normal(gen, 128, 64, std=0.1), normal(gen, 128, 64, std=0.1), normal(gen, 64, 128, std=0.1)]

    def grads(on):
        ts = [t.clone().requires_grad_(bool(o)) for t, o in zip((x, *w), on)]
        ag.gated_feed_forward(*ts).backward(dout)
        return [t.grad for t in ts]

    full = grads((1, 1, 1, 1))
    for on in ((1, 0, 0, 0), (0, 1, 1, 1), (0, 0, 1, 0), (1, 0, 0, 1)):
        for g, f, o in zip(grads(on), full, on):
            assert torch.equal(g, f) if o else g is None
    ts = [normal(gen, 9, 24).bfloat16().requires_grad_() for _ in range(2)]
    _, r = ag.rms_norm(ts[0], None, ts[1])
    r.sum().backward()  # (only the sum is used)
    assert all((t.grad == 1).all() for t in ts)


def test_inputs_off_the_boundaries_and_spaced():
    """Inputs and gradients that begin anywhere or lie apart give what dense ones give."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = normal(gen, 50, 100).bfloat16()
    w = [normal(gen, 128, 64, std=0.1).bfloat16(), normal(gen, 128, 64, std=0.1).bfloat16(), normal(gen, 64, 128, std=0.1).bfloat16()]
    for x in (wide[:, 3:67], wide[:, 8:72], wide.t()[:64].t()):
        a, b = x.detach().requires_grad_(), x.contiguous().clone().requires_grad_()
        dout = normal(gen, 50, 67).bfloat16()[:, 3:]
        oa, ob = ag.gated_feed_forward(a, *w), ag.gated_feed_forward(b, *w)
        ga, gb = torch.autograd.grad(oa, a, dout)[0], torch.autograd.grad(ob, b, dout.contiguous())[0]
        assert torch.equal(oa, ob) and torch.equal(ga, gb)
    direct = wide[:, 8:72]  # (rows 16-byte aligned, 200 bytes apart: not a multiple of 16, refused; 208: read in place)
    with pytest.raises(tb.TriAttnError):
        tb.ffn_forward(direct, *w)
    apart = torch.zeros(50, 104, dtype=torch.bfloat16, device="cuda")
    apart[:, 8:72] = direct
    assert torch.equal(tb.ffn_forward(apart[:, 8:72], *w), tb.ffn_forward(direct.contiguous(), *w))
    out, a, u = tb.ffn_forward(apart[:, 8:72], *w, keep=True)
    want = tb.ffn_backward(direct.contiguous(), *w, a, u, out)
    got = tb.ffn_backward(apart[:, 8:72], *w, a, u, out)
    assert all(torch.equal(g, e) for g, e in zip(got, want))


def _calls(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, d = normal(gen, 300, 256).bfloat16(), normal(gen, 300, 256).bfloat16()
    wg, wu, wd = normal(gen, 512, 256, std=0.06).bfloat16(), normal(gen, 512, 256, std=0.06).bfloat16(), normal(gen, 256, 512, std=0.05).bfloat16()
    _, a, u = tb.ffn_forward(x, wg, wu, wd, keep=True)
    gamma = 1 + normal(gen, 256, std=0.1)
    got = tb.rms_forward(x, gamma, d)
    table, base = normal(gen, 2 * len(STARTS), 4), normal(gen, 1, 4, 90, 90).bfloat16()
    grads = [normal(gen, n) for n in (1000, 3, 50000)]
    few = x[:5].contiguous()
    big = normal(gen, 25000, 64).bfloat16()
    wb = [normal(gen, 64, 64, std=0.1).bfloat16() for _ in range(3)]
    return {"ffn_forward": lambda s: tb.ffn_forward(x, wg, wu, wd, keep=True, stream=s), "ffn_few": lambda s: (tb.ffn_forward(few, wg, wu, wd, stream=s),),
            "ffn_block": lambda s: (tb.ffn_forward(big, *wb, stream=s),), "ffn_backward": lambda s: tb.ffn_backward(x, wg, wu, wd, a, u, d, stream=s),
            "rms_forward": lambda s: tb.rms_forward(x, gamma, d, eight_bits=True, stream=s)[:3],
            "rms_backward": lambda s: tb.rms_backward(got.r, gamma, got.rstd, d, x, stream=s),
            "relpos_forward": lambda s: (tb.relpos_forward(table, STARTS, 90, base=base, stream=s),),
            "relpos_backward": lambda s: (tb.relpos_backward(base, STARTS, stream=s),),
            "gradient_norm": lambda s: (tb.gradient_norm(grads, stream=s),)}


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_another_stream(handle):
    """A call's results and workspace may be dropped while the stream that it was given has not begun it."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for name, call in _calls().items():
        want = [t.clone() for t in call(None)]
        sizes = [t.numel() * t.element_size() for t in want] + [1 << 20, 16384]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # (about 10 ms)
        call(stream)  # (the results are dropped at once)
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        got = call(stream)
        torch.cuda.synchronize()
        assert all((o == 7).all() for o in others), name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert tb.tri_attn_device_status() == 0


def test_the_same_bits_again():
    for name, call in _calls(3).items():
        first = [t.clone() for t in call(None)]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(call(None), first)), name


def test_two_host_threads():
    """Calls of two threads on their own streams give the bits of one thread's."""
    import threading
    calls = _calls(6)
    want = {n: [t.clone() for t in c(None)] for n, c in calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    for n, c in calls.items():
                        got = c(None)
                        torch.cuda.current_stream().synchronize()
                        if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                            wrong.append(n)
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and tb.tri_attn_device_status() == 0


CHILD = """
import threading
import torch
from tests.test_feed_forward_layer_gpu import _calls
from bwd_tri_attn_gb300 import binding as tb
calls, out = _calls(100), {}
want = {n: [t.clone() for t in calls[n](None)] for n in calls}
torch.cuda.synchronize()
def work(n):
    try:
        out[n] = calls[n](None)
    except Exception as e:
        out[n] = e
for n in calls:
    t = threading.Thread(target=work, args=(n,))
    t.start()
    t.join()
    assert not isinstance(out[n], Exception), f"{n}: {out[n]}"
torch.cuda.synchronize()
for n in calls:
    assert all(torch.equal(a, b) for a, b in zip(out[n], want[n])), n
assert tb.tri_attn_device_status() == 0
"""


def test_calls_from_fresh_threads():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_rows_that_are_no_numbers_spoil_their_own():
    """An infinity or a NaN in a row of x, or in a feature's weights, stays where the formulas put it."""
    for M, C, F in ((300, 256, 512), (20000, 64, 128), (7, 128, 256)):
        gen = torch.Generator(device="cuda").manual_seed(8)
        x = normal(gen, M, C).bfloat16()
        w = [normal(gen, F, C, std=C ** -0.5).bfloat16(), normal(gen, F, C, std=C ** -0.5).bfloat16(), normal(gen, C, F, std=F ** -0.5).bfloat16()]
        want = tb.ffn_forward(x, *w, keep=True)
        bad = x.clone()
        bad[3, 5], bad[M - 1, 0] = float("nan"), float("inf")
        got = tb.ffn_forward(bad, *w, keep=True)
        rest = [i for i in (0, 2, 4, M // 2, M - 2) if i not in (3, M - 1)]
        for g, e in zip(got, want):
            assert torch.equal(g[rest], e[rest]) and not g[3].isfinite().any() and not g[M - 1].isfinite().any()
        wbad = w[0].clone()
        wbad[9, 1] = float("nan")
        _, a, u = tb.ffn_forward(x, wbad, *w[1:], keep=True)
        assert a[:, 9].isnan().all() and torch.equal(u, want[2])
        others = [f for f in range(F) if f != 9]
        assert torch.equal(a[:, others], want[1][:, others])
        dwg = tb.ffn_backward(x, wbad, *w[1:], a, u, x)[1]
        assert dwg[9].isnan().all() and dwg[others].isfinite().all()
