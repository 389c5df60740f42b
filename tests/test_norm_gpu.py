"""LayerNorm and 8-bit activation checkpoints (include/tri_norm.h) against plain 64-bit forms.

Tolerances, from the arithmetic. u is half a step of the output type (torch.finfo(t).eps / 2): one
rounding of the result. The rest is FP32 arithmetic: a row sum is at most 8 chunks of 8 values in
turn, a shuffle tree and 8 warps (under 128 roundings of 2^-24, relative to the sum of the
magnitudes), and a handful of operations follow it, so F = 2^-17 times the magnitudes that enter
an output bounds its FP32 error. A column sum adds a chunk of rows in turn (under 100 in these
tests, but for the tall case, which has its own count) and then trees: the same F times the sum of
the magnitudes. The checkpoint's format is exact: its bytes and scales must be equal.
"""
import math

import pytest
import torch

from bwd_tri_attn_gb300 import autograd as ag
from bwd_tri_attn_gb300 import binding as tb
from bwd_tri_attn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

F = 2.0 ** -17
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (rows, channels): every launch geometry, aligned and not, one row, one channel, group tails
SIZES = [(1, 1), (5, 1), (1, 8), (3, 5), (7, 64), (33, 128), (100, 130), (17, 256), (9, 384), (40, 512), (64, 768),
         (5, 1003), (3, 1024), (12, 2048), (5, 4099), (2, 8192), (3, 8191), (2000, 16), (50, 27), (61, 59), (40, 121),
         (300, 30), (700, 1003), (150, 4001), (77, 259)]


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def _normal(shape, dtype, seed, std=1.5, mean=0.25):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _weights(C, seed):
    return _normal((C,), torch.float32, seed, 0.3, 1.0), _normal((C,), torch.float32, seed + 1, 0.3, 0.0)


def _stats64(x, eps):
    x = x.double()
    mean = x.mean(-1)
    return mean, 1.0 / torch.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)


def _check_forward(x, gamma, beta, eps, y, mean, rstd):
    mu, rs = _stats64(x, eps)
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    xd = x.double()
    want = (xd - mu[..., None]) * rs[..., None] * g + b
    mag = (xd.abs() + xd.abs().mean(-1, keepdim=True)) * rs[..., None]
    # a mean off by e shifts the variance by e^2, and the sum of squares has F of its own
    assert ((mean.double() - mu).abs() <= F * xd.abs().mean(-1)).all()
    assert ((rstd.double() - rs).abs() <= (F + (F * xd.abs().mean(-1) * rs) ** 2) * rs).all()
    tol = _u(x.dtype) * want.abs() + 2 * F * (mag * (g if gamma is None else g.abs()) + (0 if beta is None else b.abs()))
    assert y.dtype == x.dtype and ((y.double() - want).abs() <= tol).all()


def _grads64(x, gamma, mean, rstd, dy):
    x, dy = x.double(), dy.double()
    g = dy if gamma is None else dy * gamma.double()
    mu, rs = mean.double()[..., None], rstd.double()[..., None]
    xh = (x - mu) * rs
    a, b = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = rs * (g - a - xh * b)
    xm = (x.abs() + mu.abs()) * rs
    mag = rs * (g.abs() + g.abs().mean(-1, keepdim=True) + xm * (g.abs() * xm).mean(-1, keepdim=True))
    rows = tuple(range(x.dim() - 1))
    return (dx, (dy * xh).sum(rows), dy.sum(rows)), (mag, (dy.abs() * xm).sum(rows), dy.abs().sum(rows))


def _check_backward(x, gamma, mean, rstd, dy, got, f=F):
    want, mag = _grads64(x, gamma, mean, rstd, dy)
    dx, dgamma, dbeta = got
    assert dx.dtype == dy.dtype and dx.shape == dy.shape
    assert ((dx.double() - want[0]).abs() <= _u(dy.dtype) * want[0].abs() + 2 * f * mag[0]).all()
    for w, m, t in zip(want[1:], mag[1:], (dgamma, dbeta)):
        assert t.dtype == torch.float32 and ((t.double() - w).abs() <= 2 * f * m).all()


def _values(x):
    """The checkpoint's bytes, scales and values by its definition, for finite x."""
    C = x.shape[-1]
    n = (C + 127) // 128
    g = torch.nn.functional.pad(x.float(), (0, n * 128 - C)).unflatten(-1, (n, 128))
    top = g.abs().amax(-1)
    most = torch.full_like(top, 127.0)
    live = top >= 2.0 ** -120
    s = torch.where(live, top / most, torch.zeros_like(top))
    s = torch.where((s * most).isinf(), torch.nextafter(s, torch.zeros_like(s)), s)  # 127 s stays finite
    inv = torch.where(live, most / top, torch.zeros_like(top))
    q = torch.round(g * inv[..., None])
    return q.flatten(-2)[..., :C].to(torch.int8), s, (q * s[..., None]).flatten(-2)[..., :C]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M,C", SIZES)
def test_forward_backward_and_checkpoint(M, C, dtype):
    x, dy = _normal((M, C), dtype, 1), _normal((M, C), dtype, 2, 1.0, 0.0)
    gamma, beta = _weights(C, 3)
    y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
    y2, mean2, rstd2 = tb.norm_forward(x, gamma, beta)
    got = tb.norm_backward(x, gamma, mean, rstd, dy)
    from_kept = tb.norm_backward(kept, gamma, mean, rstd, dy)
    packed = tb.checkpoint_pack(x)
    back = tb.checkpoint_unpack(packed, dtype=dtype)
    torch.cuda.synchronize()
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    _check_backward(x, gamma, mean, rstd, dy, got)
    q, s, v = _values(x)
    for k in (kept, packed):
        assert torch.equal(k.q8, q) and torch.equal(k.scale, s)
    assert torch.equal(back, v.to(dtype))
    _check_backward(v, gamma, mean, rstd, dy, from_kept)


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
def test_without_weights(gamma, beta):
    x, dy = _normal((37, 96), torch.bfloat16, 5), _normal((37, 96), torch.bfloat16, 6, 1.0, 0.0)
    g, b = _weights(96, 7)
    g, b = (g if gamma else None), (b if beta else None)
    y, mean, rstd = tb.norm_forward(x, g, b)
    got = tb.norm_backward(x, g, mean, rstd, dy)
    _check_forward(x, g, b, 1e-5, y, mean, rstd)
    if gamma:
        _check_backward(x, g, mean, rstd, dy, got)
    else:
        assert got[1] is None and got[2] is None
        want, mag = _grads64(x, None, mean, rstd, dy)
        assert ((got[0].double() - want[0]).abs() <= 2.0 ** -8 * want[0].abs() + 2 * F * mag[0]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("C,width,start", [(128, 160, 16), (128, 160, 3), (100, 101, 0), (1000, 2048, 1)])
def test_spaced_and_unaligned_rows(C, width, start, dtype):
    """Rows that are part of wider ones (row strides, starts off the 16-byte boundaries), of a 3-D tensor."""
    wide, dwide = _normal((4, 9, width), dtype, 8), _normal((4, 9, width), dtype, 9, 1.0, 0.0)
    x, dy = wide[..., start:start + C], dwide[..., start:start + C]
    gamma, beta = _weights(C + 1, 10)
    gamma, beta = gamma[1:], beta[1:]  # 4-byte alignment only
    y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
    got = tb.norm_backward(x, gamma, mean, rstd, dy)
    packed = tb.checkpoint_pack(x)
    assert y.is_contiguous() and y.shape == x.shape and mean.shape == x.shape[:-1]
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_backward(x, gamma, mean, rstd, dy, got)
    q, s, _ = _values(x)
    for k in (kept, packed):
        assert torch.equal(k.q8, q) and torch.equal(k.scale, s)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("M,C,off", [(50, 259, 3), (9, 64, 1), (300, 1001, 2)])
def test_backward_into_buffers_equally_far_from_a_boundary(M, C, off, dtype):
    """x, dy and dx (and the checkpoint) that start the same number of values behind a 16-byte boundary; nothing is
    written before or behind dx."""
    x, dy = _normal((M, C), dtype, 20), _normal((M, C), dtype, 21, 1.0, 0.0)
    gamma, _ = _weights(C, 22)
    _, mean, rstd, kept = tb.norm_forward(x, gamma, checkpoint=True)
    vec = 16 // x.element_size()
    shape = tb.norm_shape_of(x, dy=dy)
    ws = torch.empty(tb.tri_norm_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")

    def shifted(t):
        wide = torch.full((t.numel() + 2 * vec,), 7, dtype=t.dtype, device="cuda")
        part = wide[off:off + t.numel()].view(t.shape)
        part.copy_(t)
        return wide, part

    (_, xs), (_, ds), (wide, dx), (_, q8) = shifted(x), shifted(dy), shifted(x), shifted(kept.q8)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
    for eight_bits in (False, True):
        wide.fill_(7)
        tb.tri_norm_bwd(shape, None if eight_bits else xs, q8 if eight_bits else None, kept.scale if eight_bits else None, gamma,
                        mean, rstd, ds, dx, dgamma, dbeta, ws)
        assert (wide[:off] == 7).all() and (wide[off + M * C:] == 7).all()
        _check_backward(tb.checkpoint_unpack(kept, torch.float32) if eight_bits else x, gamma, mean, rstd, dy, (dx, dgamma, dbeta))


def test_rows_far_from_zero():
    """A common offset of 1000: the variance is of the differences, not a difference of squares."""
    x = _normal((50, 384), torch.float32, 11, 0.5, 1000.0)
    gamma, beta = _weights(384, 12)
    y, mean, rstd = tb.norm_forward(x, gamma, beta)
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)


def test_tall():
    """More rows than one pass of the forward grid; 72 rows a lane group in the column sums."""
    x, dy = _normal((700001, 128), torch.bfloat16, 13), _normal((700001, 128), torch.bfloat16, 14, 1.0, 0.0)
    gamma, beta = _weights(128, 15)
    y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
    got = tb.norm_backward(x, gamma, mean, rstd, dy)
    _check_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_backward(x, gamma, mean, rstd, dy, got)
    q, s, _ = _values(x)
    assert torch.equal(kept.q8, q) and torch.equal(kept.scale, s)
    packed = tb.checkpoint_pack(x)
    assert torch.equal(packed.q8, q) and torch.equal(packed.scale, s)


def test_constant_rows():
    x = torch.full((6, 256), 3.0, device="cuda", dtype=torch.bfloat16)
    gamma, beta = _weights(256, 16)
    y, mean, rstd = tb.norm_forward(x, gamma, beta)
    assert torch.equal(mean, torch.full_like(mean, 3.0))
    assert torch.equal(y, beta.to(torch.bfloat16).expand(6, 256))
    assert ((rstd.double() - 1 / math.sqrt(1e-5)).abs() <= F / math.sqrt(1e-5)).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_checkpoint_of_unusual_values(dtype):
    x = _normal((8, 300), dtype, 17)
    x[0, :128] = 0.0                                    # a group of zeros beside others
    x[1, 5] = math.inf                                  # comes back as NaN, its own group alone
    x[2, 130] = -math.inf
    x[3, 299] = math.nan
    x[4] = 0.0
    x[4, 7] = torch.finfo(dtype).max                    # one value alone keeps to FP32 rounding
    x[5] = torch.finfo(dtype).tiny if dtype == torch.float32 else torch.finfo(torch.float16).tiny
    x[6, :128] = torch.tensor([(-1.0) ** k for k in range(128)], dtype=dtype, device="cuda")
    kept = tb.checkpoint_pack(x)
    back = tb.checkpoint_unpack(kept, dtype=torch.float32)
    _, _, _, kept2 = tb.norm_forward(x, checkpoint=True)
    assert torch.equal(kept.q8, kept2.q8) and torch.equal(kept.scale.isnan(), kept2.scale.isnan())
    nan = torch.zeros((8, 300), dtype=torch.bool, device="cuda")
    nan[1, :128] = nan[2, 128:256] = nan[3, 256:] = True
    assert torch.equal(back.isnan(), nan)
    fine = x.clone()
    fine[nan] = 0.0
    q, s, v = _values(fine)
    assert torch.equal(torch.where(nan, torch.zeros_like(v), back), v)
    assert torch.equal(back[6, :128], x[6, :128].float())
    top = torch.finfo(dtype).max
    assert abs(back[4, 7].item() - top) <= 2.0 ** -22 * top
    # within half a step of a group's scale, and a quarter of an FP32 rounding of the product's
    step = s.repeat_interleave(128, -1)[:, :300]
    assert ((v - fine.float()).abs() <= 0.5 * step * (1 + 2.0 ** -15) + (step == 0) * 2.0 ** -120).all()


def test_gradient_against_differences():
    """Central differences of sum(w y) in 64 bits at the formula, step 1e-4, against the kernel's FP32 gradients:
    the difference's own error is under 1e-6 of the gradient's scale, the kernel's under F."""
    x, w = _normal((3, 40), torch.float32, 18), _normal((3, 40), torch.float32, 19, 1.0, 0.0)
    gamma, beta = _weights(40, 20)
    _, mean, rstd = tb.norm_forward(x, gamma, beta)
    dx, dgamma, dbeta = tb.norm_backward(x, gamma, mean, rstd, w)

    def loss(xd, g, b):
        mu, rs = _stats64(xd, 1e-5)
        return (((xd - mu[:, None]) * rs[:, None] * g + b) * w.double()).sum()

    h = 1e-4
    args = [x.double(), gamma.double(), beta.double()]
    for k, grad in enumerate((dx, dgamma, dbeta)):
        flat = args[k].reshape(-1)
        for i in range(0, flat.numel(), 7):
            lo, hi = ([a.clone() for a in args] for _ in range(2))
            lo[k].reshape(-1)[i] -= h
            hi[k].reshape(-1)[i] += h
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(diff.item() - grad.reshape(-1)[i].item()) <= 1e-4 * max(1.0, abs(diff.item()))


def test_same_bits_in_a_graph_and_on_another_stream():
    x, dy = _normal((4100, 200), torch.bfloat16, 21), _normal((4100, 200), torch.bfloat16, 22, 1.0, 0.0)
    gamma, beta = _weights(200, 23)

    def step():
        y, mean, rstd, kept = tb.norm_forward(x, gamma, beta, checkpoint=True)
        return (y, mean, rstd, *kept, *tb.norm_backward(x, gamma, mean, rstd, dy),
                *tb.norm_backward(kept, gamma, mean, rstd, dy), tb.checkpoint_unpack(kept))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        for t in captured:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("weights", [torch.float32, torch.bfloat16, None], ids=str)
def test_autograd(checkpoint, weights):
    x = _normal((2, 30, 96), torch.bfloat16, 24).requires_grad_(True)
    dy = _normal((2, 30, 96), torch.bfloat16, 25, 1.0, 0.0)
    g = b = None
    if weights is not None:
        g, b = (t.to(weights).requires_grad_(True) for t in _weights(96, 26))
    y = ag.layer_norm(x, g, b, 1e-3, checkpoint)
    y.backward(dy)
    g32, b32 = (None if t is None else t.detach().float() for t in (g, b))
    out = tb.norm_forward(x.detach(), g32, b32, eps=1e-3, checkpoint=checkpoint)
    want = tb.norm_backward(out[3] if checkpoint else x.detach(), g32, out[1], out[2], dy)
    assert torch.equal(y, out[0]) and torch.equal(x.grad, want[0])
    if weights is not None:
        assert torch.equal(g.grad, want[1].to(weights)) and torch.equal(b.grad, want[2].to(weights))


def test_autograd_beta_alone():
    x = _normal((30, 96), torch.bfloat16, 27).requires_grad_(True)
    b = _weights(96, 28)[1].requires_grad_(True)
    dy = _normal((30, 96), torch.bfloat16, 29, 1.0, 0.0)
    ag.layer_norm(x, None, b).backward(dy)
    assert ((b.grad.double() - dy.double().sum(0)).abs() <= F * dy.double().abs().sum(0)).all()


def test_block_keeps_its_input_in_8_bits():
    """The triangle-attention block with a checkpoint: the forward pass is the plain one's bit for bit, the
    gradients are bitwise those of the block at the checkpoint's values, and far less memory lives in between."""
    torch.manual_seed(0)
    m = ag.TriangleAttentionBlock(c=128, H=4, d=32, device="cuda")
    k = ag.TriangleAttentionBlock(c=128, H=4, d=32, device="cuda", checkpoint=True)
    k.load_state_dict(m.state_dict())
    x = wl.make_module_inputs(1, 72, 128, 4, 32, seed=81, mask=("tail", 3))
    mask, dout = x["mask"].cuda(), x["dout"].cuda()

    def run(block, z):
        z = z.clone().requires_grad_(True)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = block(z, mask)
        held = torch.cuda.memory_allocated() - before
        out.backward(dout)
        return out.detach(), held, (z.grad, *(p.grad for p in block.parameters()))

    z = x["z"].cuda()
    plain, held_plain, _ = run(m, z)
    out, held, grads = run(k, z)
    m.zero_grad()
    values = tb.checkpoint_unpack(tb.checkpoint_pack(z))
    _, _, want = run(m, values)
    assert torch.equal(out, plain)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    # besides out (2 c bytes a position, in both): 1 + 1/32 bytes a value against zt (2 c bytes a position)
    # and q, k, v, gate, O, its residual and the gated output (seven times 2 H d, H d = 128)
    pos, c = 72 * 72, 128
    assert held <= pos * (2 * c + c + 4) + (1 << 20) and held_plain >= pos * (2 * c + 2 * c + 14 * 128)
