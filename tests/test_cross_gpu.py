"""Cross attention (include/tri_cross.h) against a plain 64-bit form, through the public binding.

Tolerances, from the arithmetic. U = 2^-8 is half a step of BF16: one rounding of every output, one of
every P (forward, dV) and dS (dQ, dK) before the second product. The rest is FP32: a score is a sum
of d products, off by at most d 2^-24 of scale sum |q k| before the exponential and by a few units of
2^-24 of its own and LSE's magnitude in the exponent, so a probability is off by the relative E below; a
row of dP and D are sums of d products each (2^-16 of their magnitudes covers d = 128 roundings). Sums over keys
and queries are FP32 with fewer than 2^-16 in all, relative to the sum of the magnitudes, in these tests.
"""
import math

import pytest
import torch

from bwd_tri_attn_gb300 import autograd as ag
from bwd_tri_attn_gb300 import binding as tb

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -16


def make(B, T, S, H, Hk, d, lens=None, mask=None, seed=0, layout="dense"):
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + 7)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    x = {"q": normal(B, T, H, d), "do": normal(B, T, H, d)}
    if layout == "fused":  # keys and values from one projection, queries a part of wider rows
        kv = normal(B, S, 2, Hk, d)
        x["k"], x["v"] = kv[:, :, 0], kv[:, :, 1]
        x["q"] = normal(B, T, H, d + 16)[..., 8:d + 8]
    elif layout == "heads":  # heads before positions
        x["q"] = normal(B, H, T, d).transpose(1, 2)
        x["k"], x["v"] = normal(B, Hk, S, d).transpose(1, 2), normal(B, Hk, S, d).transpose(1, 2)
    else:
        x["k"], x["v"] = normal(B, S, Hk, d), normal(B, S, Hk, d)
    x["lens"] = None
    if lens is not None:
        x["lens"] = torch.tensor([lens[b % len(lens)] for b in range(B)], dtype=torch.int32, device="cuda")
    x["mask"] = None
    if mask is not None:
        m = torch.rand((B, S), generator=gen, device="cuda") < mask
        m[0] = m[0] & (torch.arange(S, device="cuda") // 128 != 1)  # a whole tile without live keys
        if B > 2:
            m[2] = False  # a sequence without live keys
        x["mask"] = m
    return x


def live_keys(x):
    B, S = x["k"].shape[:2]
    live = torch.ones((B, S), dtype=torch.bool, device="cuda")
    if x["lens"] is not None:
        live &= torch.arange(S, device="cuda") < x["lens"][:, None]
    if x["mask"] is not None:
        live &= x["mask"].bool()
    return live


def heads64(t, group=1):
    return t.double().transpose(1, 2).repeat_interleave(group, 1)


def oracle(x, scale, o=None, lse=None):
    """Every output and its tolerance, [B, heads, n, d]; with o and lse the backward pass at them."""
    q, group = heads64(x["q"]), x["q"].shape[2] // x["k"].shape[2]
    live = live_keys(x)
    clean = live[:, :, None, None]
    k, v = (heads64(torch.where(clean, x[n], torch.zeros_like(x[n])), group) for n in ("k", "v"))
    dead = ~live[:, None, None]
    s = (q @ k.transpose(2, 3) * scale).masked_fill(dead, -math.inf)
    mag = q.abs() @ k.abs().transpose(2, 3) * abs(scale)
    if o is None:
        want_lse = torch.logsumexp(s, -1)
        at = want_lse
    else:
        at = lse.double()
    p = torch.exp(s - torch.where(at == -math.inf, torch.zeros_like(at), at)[..., None])
    E = F * (mag + at.abs().nan_to_num(posinf=0.0)[..., None] + 1.0)
    if o is None:
        ev = (p * (U + 2 * E)) @ v.abs()
        want = p @ v
        tl = F * (mag.masked_fill(dead, 0.0).amax(-1) + want_lse.abs().nan_to_num(posinf=0.0) + 1.0)
        return {"O": (want, U * want.abs() + ev + 1e-30), "LSE": (want_lse, tl)}
    do, ob = heads64(x["do"]), heads64(o)
    delta = (do * ob).sum(-1, keepdim=True)
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - delta)
    ds_err = ds.abs() * (U + 2 * E) + p * F * (do.abs() @ v.abs().transpose(2, 3) + (do * ob).abs().sum(-1, keepdim=True))
    dq, dk, dv = ds @ k * scale, ds.transpose(2, 3) @ q * scale, p.transpose(2, 3) @ do
    eq, ek = ds_err @ k.abs() * abs(scale), ds_err.transpose(2, 3) @ q.abs() * abs(scale)
    ev = (p * (U + 2 * E)).transpose(2, 3) @ do.abs()

    def shared(t):
        return t.unflatten(1, (-1, group)).sum(2)

    out = {"dQ": (dq, eq), "dK": (shared(dk), shared(ek)), "dV": (shared(dv), shared(ev))}
    return {n: (w, U * w.abs() + e + 1e-30) for n, (w, e) in out.items()}


def close(name, got, want_tol, transposed=True):
    want, tol = want_tol
    g = got.double().transpose(1, 2) if transposed else got.double()
    inf = want.isinf()
    assert torch.equal(g.isinf(), inf) and torch.equal(g[inf], want[inf]), name
    err = (g - want).masked_fill(inf, 0.0).abs()
    assert (err <= tol).all(), f"{name}: {(err / tol.clamp_min(1e-300)).max().item():.3f} of the tolerance"


def check(x, scale=None, backward=True):
    d = x["q"].shape[3]
    at = d ** -0.5 if scale is None else scale
    O, LSE = tb.cross_forward(x["q"], x["k"], x["v"], x["mask"], x["lens"], scale)
    assert tb.tri_attn_device_status() == 0
    for name, w in oracle(x, at).items():
        close(name, O if name == "O" else LSE, w, name == "O")
    if not backward:
        return O, LSE
    got = tb.cross_backward(x["q"], x["k"], x["v"], O, LSE, x["do"], x["mask"], x["lens"], scale)
    assert tb.tri_attn_device_status() == 0
    ref = oracle(x, at, O, LSE)
    for name, g in zip(("dQ", "dK", "dV"), got):
        close(name, g, ref[name])
    return (O, LSE, *got)


SIZES = [  # B, T, S, H, Hk, d
    (1, 1, 1, 1, 1, 8), (1, 16, 77, 4, 4, 32), (2, 1, 2, 2, 1, 16), (1, 127, 129, 2, 2, 64), (1, 128, 128, 1, 1, 128),
    (2, 129, 127, 2, 1, 40), (1, 257, 513, 3, 3, 72), (3, 33, 300, 6, 2, 24), (1, 300, 1100, 4, 2, 128), (2, 5, 640, 16, 2, 80),
    (1, 3, 200, 128, 1, 64), (1, 2, 140, 160, 1, 32), (1, 700, 257, 2, 2, 96), (5, 1, 1000, 12, 4, 120), (2, 520, 1030, 8, 4, 64),
]


@pytest.mark.parametrize("B,T,S,H,Hk,d", SIZES)
def test_sizes(B, T, S, H, Hk, d):
    check(make(B, T, S, H, Hk, d, seed=1))


@pytest.mark.parametrize("layout", ["fused", "heads"])
@pytest.mark.parametrize("B,T,S,H,Hk,d", [(2, 150, 300, 4, 2, 64), (3, 1, 300, 8, 8, 128), (1, 130, 1, 2, 1, 40)])
def test_strides(B, T, S, H, Hk, d, layout):
    x = make(B, T, S, H, Hk, d, seed=2, layout=layout)
    got = check(x)
    dense = dict(x, **{n: x[n].contiguous() for n in "qkv"})
    for a, b in zip(got, check(dense)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[0], [1], [128], [127, 129, 0], [300, 1, 256, 17]])
@pytest.mark.parametrize("T,H,Hk,d", [(1, 8, 2, 64), (140, 2, 2, 128)])
def test_lengths(lens, T, H, Hk, d):
    check(make(4, T, 300, H, Hk, d, lens=lens, seed=3))


@pytest.mark.parametrize("S,mask,lens", [(300, 0.5, None), (513, 0.02, None), (400, 0.9, [400, 0, 129, 1])])
@pytest.mark.parametrize("T,H,Hk,d", [(1, 4, 1, 128), (200, 4, 2, 32)])
def test_masks(S, mask, lens, T, H, Hk, d):
    x = make(4, T, S, H, Hk, d, lens=lens, mask=mask, seed=4)
    a = check(x)
    b = check(dict(x, mask=x["mask"].to(torch.uint8) * 7))
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).max])
def test_dead_keys_may_hold_anything(bad):
    x = make(4, 140, 400, 4, 2, 64, lens=[400, 0, 129, 250], mask=0.8, seed=5)
    a = check(x)
    dead = ~live_keys(x)
    b = check(dict(x, k=x["k"].masked_fill(dead[:, :, None, None], bad), v=x["v"].masked_fill(dead[:, :, None, None], bad)))
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_lengths_outside_the_range_are_clamped():
    x = make(3, 20, 200, 2, 2, 32, lens=[200, 0, 130], seed=6)
    a = check(x)
    y = dict(x, lens=torch.tensor([2 ** 31 - 1, -5, 130], dtype=torch.int32, device="cuda"))
    O, LSE = tb.cross_forward(y["q"], y["k"], y["v"], None, y["lens"])
    got = tb.cross_backward(y["q"], y["k"], y["v"], O, LSE, y["do"], None, y["lens"])
    for s, t in zip(a, (O, LSE, *got)):
        assert torch.equal(s, t)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 3e-5])
def test_scales(scale):
    check(make(2, 70, 300, 4, 2, 64, mask=0.9, seed=7), scale=scale)


def test_growing_scores():
    """Scores that rise along the keys: the running maximum moves at every tile, by far more than the rescaling threshold."""
    x = make(1, 200, 1500, 2, 2, 64, seed=8)
    ramp = torch.linspace(0.0, 6.0, 1500, device="cuda")[None, :, None, None]
    x["q"], x["k"] = (x["q"].float().abs()).bfloat16(), (x["k"].float().abs() * ramp).bfloat16()
    check(x)
    x["k"] = x["k"].flip(1)
    check(x)


def test_many_sequences():
    """More sequences than a warp's lanes, lengths from 0 up: the search for a CTA's first unit."""
    check(make(70, 3, 260, 2, 1, 32, lens=list(range(0, 261, 4)), seed=9))


def test_long_keys():
    """One query of each sequence, keys split over many CTAs."""
    check(make(2, 1, 20000, 8, 2, 128, lens=[20000, 9000], seed=10))


def test_offsets_past_32_bits():
    """Encoder states of more than 2^31 elements, a view into a larger buffer; checked on slices of its keys."""
    S, Hk, d = 1 << 21, 8, 128
    buf = torch.empty((1, S, 2, Hk, d), dtype=torch.bfloat16, device="cuda").normal_()
    k, v = buf[:, :, 0], buf[:, :, 1]
    q = torch.randn(1, 1, Hk, d, device="cuda").bfloat16()
    mask = torch.zeros((1, S), dtype=torch.bool, device="cuda")
    keep = torch.tensor([0, 5, (1 << 20) + 3, S - 130, S - 1], device="cuda")
    mask[0, keep] = True
    O, LSE = tb.cross_forward(q, k, v, mask)
    want = tb.cross_forward(q, k[:, keep].contiguous(), v[:, keep].contiguous())
    torch.cuda.synchronize()
    x = {"q": q, "k": k[:, keep], "v": v[:, keep], "lens": None, "mask": None}
    for got in ((O, LSE), want):
        for name, w in oracle(x, d ** -0.5).items():
            close(name, got[0] if name == "O" else got[1], w, name == "O")


def test_against_differences():
    """Central differences of sum(w O) at the 64-bit formula. The kernel's D is from the BF16 O: off by U sum |w O|,
    which moves dS by p times that; everything else is in the formula's own tolerance."""
    x = make(1, 4, 9, 2, 1, 8, seed=11)
    w = heads64(x["do"])
    scale = 8 ** -0.5
    O, LSE, dQ, dK, dV = check(x)

    def loss(q, k, v):
        s = q @ k.repeat_interleave(2, 1).transpose(2, 3) * scale
        return (torch.softmax(s, -1) @ v.repeat_interleave(2, 1) * w).sum()

    args = [heads64(x[n]) for n in "qkv"]
    tol = {n: t[1] for n, t in oracle(x, scale, O, LSE).items()}
    p = torch.softmax(args[0] @ args[1].repeat_interleave(2, 1).transpose(2, 3) * scale, -1)
    dd = p * (2 * U * (w * heads64(O)).abs().sum(-1, keepdim=True)) * scale
    extra = [dd @ args[1].repeat_interleave(2, 1).abs(),
             (dd.transpose(2, 3) @ args[0].abs()).unflatten(1, (-1, 2)).sum(2), torch.zeros_like(args[2])]
    h = 1e-5
    for a, (name, got) in enumerate((("dQ", dQ), ("dK", dK), ("dV", dV))):
        got, lim = got.double().transpose(1, 2), tol[name] + extra[a] + 1e-7
        flat = args[a].reshape(-1)
        for i in range(flat.numel()):
            lo, hi = ([t.clone() for t in args] for _ in range(2))
            lo[a].reshape(-1)[i] -= h
            hi[a].reshape(-1)[i] += h
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(diff - got.reshape(-1)[i]) <= lim.reshape(-1)[i], (name, i)


def test_same_bits_in_a_graph_and_on_another_stream():
    x = make(3, 200, 900, 8, 2, 64, lens=[900, 400, 0], mask=0.9, seed=12)

    def step():
        O, LSE = tb.cross_forward(x["q"], x["k"], x["v"], x["mask"], x["lens"])
        return (O, LSE, *tb.cross_backward(x["q"], x["k"], x["v"], O, LSE, x["do"], x["mask"], x["lens"]))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)
    # replayed with other lengths: they are read on the device
    x["lens"].copy_(torch.tensor([1, 0, 900], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, step()):
        assert torch.equal(a, b)
    assert tb.tri_attn_device_status() == 0


def test_two_streams_at_once():
    """Two calls in flight together, each with its own workspace (both want every SM and its tensor memory)."""
    xs = [make(2, 300, 1500, 4, 4, 128, seed=13), make(2, 300, 1500, 4, 4, 128, lens=[700, 1500], seed=14)]
    want = [check(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                O, LSE = tb.cross_forward(x["q"], x["k"], x["v"], None, x["lens"])
                got[i].append((O, LSE, *tb.cross_backward(x["q"], x["k"], x["v"], O, LSE, x["do"], None, x["lens"])))
    torch.cuda.synchronize()
    assert tb.tri_attn_device_status() == 0
    for i in range(2):
        for g in got[i]:
            for a, b in zip(want[i], g):
                assert torch.equal(a, b)


def test_autograd():
    x = make(2, 100, 260, 4, 2, 64, lens=[260, 30], mask=0.9, seed=15, layout="heads")
    q, k, v = (x[n].clone().requires_grad_(True) for n in "qkv")
    O = ag.cross_attention(q, k, v, x["mask"], x["lens"])
    O.backward(x["do"].transpose(1, 2).contiguous().transpose(1, 2))
    want = check(x)
    assert torch.equal(O.detach(), want[0])
    for t, g in zip((q, k, v), want[2:]):
        assert torch.equal(t.grad, g)
    q2 = q.detach().requires_grad_(True)
    (g,) = torch.autograd.grad(ag.cross_attention(q2, k.detach(), v.detach()), q2, x["do"], create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_workspace_of_the_wrong_size():
    x = make(1, 200, 900, 4, 4, 64, seed=16)
    shape = tb.cross_shape_of(x["q"], x["k"], x["v"])
    O, LSE = tb.cross_forward(x["q"], x["k"], x["v"])
    for size, call in ((tb.tri_cross_fwd_workspace_size(shape), lambda ws: tb.cross_forward(x["q"], x["k"], x["v"], workspace=ws)),
                       (tb.tri_cross_bwd_workspace_size(shape),
                        lambda ws: tb.cross_backward(x["q"], x["k"], x["v"], O, LSE, x["do"], workspace=ws))):
        assert size > 16
        with pytest.raises(tb.TriAttnError) as e:
            call(torch.empty(size - 16, dtype=torch.uint8, device="cuda"))
        assert e.value.code == -3
        call(torch.empty(size, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert tb.tri_attn_device_status() == 0
