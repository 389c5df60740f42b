"""PyTorch autograd glue over the C ABI (argument marshalling only).

Every forward and backward step runs in the library's kernels through ``binding``; these classes
only keep the tensors the backward pass needs and hand gradients back in the dtypes autograd
expects. There is no CPU path: the library raises if it is missing or a call fails. Inputs and
gradients are made contiguous, and copied to a 16-byte boundary where the library wants one (a no-op
for fresh tensors); dtypes and sizes are checked by the binding. The backward passes are
differentiable once (no second derivatives); forward-mode derivatives are refused.

- ``triangle_attention(Q, K, V, bias, mask=None, node=NODE_STARTING)``: the attention core
  (include/tri_attn.h) with its residual-compensated backward; gradients for Q, K, V and bias.
- ``triangle_multiplication(Pa, Ga, Pb, Gb, incoming=False, layout=LAYOUT_PAIR)``: the triangle
  multiplicative update (include/tri_mul.h); X channel-major [B, C, N, N], gradients for the four
  projections in their layout.
- ``triangle_attention_block(z, gamma, beta, W, wb, Wo, mask, H, d, node, eps)`` and
  ``TriangleAttentionBlock``: the surrounding block (include/tri_module.h). The weights may be FP32
  masters: the forward uses their BF16 rounding (as mixed-precision training does) and the
  backward returns the library's FP32 weight gradients in the masters' dtype. With ``checkpoint``
  the block keeps its input in 8 bits and recomputes.
- ``layer_norm(x, gamma, beta, eps, checkpoint=False)``: LayerNorm (include/tri_norm.h), gradients
  for x and the weights; with ``checkpoint`` it keeps x in 8 bits for the backward pass.
- ``cross_attention(Q, K, V, mask=None, kv_lens=None, scale=None)``: cross attention to an encoder's
  states of another length (include/tri_cross.h), gradients for Q, K and V.
- ``relative_position_bias(table, starts, Nq, ...)``: the pair bias from a learned table of distances
  (include/tri_relpos.h), gradients for the table and the base.
- ``rms_norm(x, gamma=None, residual=None, eps=1e-5)``: RMS norm, with the residual's addition
  (include/tri_rms.h).
- ``gated_feed_forward(x, Wg, Wu, Wd, act, checkpoint=False)``: the gated feed-forward block
  (include/tri_ffn.h), weights as in the block above; ``feed_forward_layer`` and ``FeedForwardLayer``: it
  behind the norm of a residual sum.
- ``clip_grad_norm_(parameters, max_norm)``: clips gradients in place to a norm of all of them together
  (include/tri_clip.h).
"""
from __future__ import annotations

import math

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import binding as tb


def _dense(t):
    """t contiguous from a 16-byte boundary on: t itself where it is (a contiguous view, such as a concatenation's
    gradient, may begin anywhere), else a copy."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _TriangleAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, bias, mask, node):
        Q, K, V, bias = (_dense(t) for t in (Q, K, V, bias))
        mask = None if mask is None else _dense(mask)
        O, LSE, Ores = tb.forward(Q, K, V, bias, mask, node=node)
        ctx.node = node
        ctx.save_for_backward(Q, K, V, bias, mask, O, Ores, LSE)
        return O

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        Q, K, V, bias, mask, O, Ores, LSE = ctx.saved_tensors
        dQ, dK, dV, dBias = tb.backward(Q, K, V, bias, mask, O, Ores, LSE,
                                        _dense(dO.to(torch.bfloat16)), node=ctx.node)
        return dQ, dK, dV, dBias, None, None


def triangle_attention(Q, K, V, bias, mask=None, node=tb.NODE_STARTING):
    """O of the attention core for BF16 CUDA tensors Q, K, V [B, S, N, H, d] (starting node; the
    ending node takes [B, N, S, H, d] in place), bias [B, H, N, N], mask [B, S, N] or None."""
    return _TriangleAttention.apply(Q, K, V, bias, mask, node)


class _TriangleMultiplication(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Pa, Ga, Pb, Gb, incoming, layout):
        Pa, Ga, Pb, Gb = (_dense(t) for t in (Pa, Ga, Pb, Gb))
        X, A, Bm = tb.mul_forward(Pa, Ga, Pb, Gb, incoming=incoming, layout=layout)
        ctx.cfg = (incoming, layout)
        ctx.save_for_backward(Pa, Ga, Pb, Gb, A, Bm)
        return X

    @staticmethod
    @once_differentiable
    def backward(ctx, dX):
        Pa, Ga, Pb, Gb, A, Bm = ctx.saved_tensors
        incoming, layout = ctx.cfg
        grads = tb.mul_backward(Pa, Ga, Pb, Gb, A, Bm, _dense(dX.to(torch.bfloat16)), incoming=incoming,
                                layout=layout)
        return (*grads, None, None)


def triangle_multiplication(Pa, Ga, Pb, Gb, incoming=False, layout=tb.LAYOUT_PAIR):
    """X [B, C, N, N] of the triangle multiplicative update for BF16 CUDA projections and gate
    logits (layout LAYOUT_PAIR: [B, N, N, C]; LAYOUT_CHANNEL_MAJOR: [B, C, N, N])."""
    return _TriangleMultiplication.apply(Pa, Ga, Pb, Gb, incoming, layout)


class _TriangleAttentionBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, gamma, beta, W, wb, Wo, mask, H, d, node, eps, checkpoint):
        z = _dense(z)
        mask = None if mask is None else _dense(mask)
        bf = [_dense(t.to(torch.bfloat16)) for t in (W, wb, Wo)]
        g32, b32 = _dense(gamma.float()), _dense(beta.float())
        out, saved = tb.module_forward(z, g32, b32, *bf, mask, H, d, node=node, eps=eps)
        ctx.meta = (H, d, node, eps, [t.dtype for t in (gamma, beta, W, wb, Wo)])
        ctx.kept_in_8_bits = checkpoint
        ctx.save_for_backward(g32, b32, *bf, mask, *(tb.checkpoint_pack(z) if checkpoint else (z, saved)))
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        g32, b32, W, wb, Wo, mask, *kept = ctx.saved_tensors
        H, d, node, eps, dtypes = ctx.meta
        if ctx.kept_in_8_bits:
            z = tb.checkpoint_unpack(kept)
            _, saved = tb.module_forward(z, g32, b32, W, wb, Wo, mask, H, d, node=node, eps=eps)
        else:
            z, saved = kept
        grads = tb.module_backward(z, g32, b32, W, wb, Wo, mask, saved, _dense(dout.to(torch.bfloat16)),
                                   H, d, node=node, eps=eps)
        dz = grads[0]
        wgrads = [g.to(dt) for g, dt in zip(grads[1:], dtypes)]
        return (dz, *wgrads, None, None, None, None, None, None)


def triangle_attention_block(z, gamma, beta, W, wb, Wo, mask, H, d, node=tb.NODE_STARTING, eps=1e-5,
                             checkpoint=False):
    """The triangle-attention block on the BF16 pair representation z [B, N, N, c]: LayerNorm
    (gamma, beta [c]), projections W [4 H d, c] (q, k, v, gate rows) and wb [H, c], the attention,
    the sigmoid gate and the output projection Wo [c, H d].

    With ``checkpoint`` the block keeps z in 8 bits (one byte and 1/32 of an FP32 scale a value) in
    the place of z and its activations (at least 4 c + 14 H d bytes a pair position), and the backward
    pass recomputes them: its gradients are those of the block at the checkpoint's values of z."""
    return _TriangleAttentionBlock.apply(z, gamma, beta, W, wb, Wo, mask, H, d, node, eps, checkpoint)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps, checkpoint):
        x = x.contiguous()
        g32, b32 = (None if t is None else t.float().contiguous() for t in (gamma, beta))
        y, mean, rstd, *kept = tb.norm_forward(x, g32, b32, eps=eps, checkpoint=checkpoint)
        ctx.kept_in_8_bits = checkpoint
        ctx.dtypes = tuple(None if t is None else t.dtype for t in (gamma, beta))
        ctx.save_for_backward(g32, mean, rstd, *(kept[0] if checkpoint else (x,)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        g32, mean, rstd, *kept = ctx.saved_tensors
        x = tb.Checkpoint(*kept) if ctx.kept_in_8_bits else kept[0]
        if g32 is None and ctx.dtypes[1] is not None:  # (beta alone: its gradient is taken with gamma = 1)
            g32 = torch.ones(dy.shape[-1], dtype=torch.float32, device=dy.device)
        grads = tb.norm_backward(x, g32, mean, rstd, dy.contiguous())
        wgrads = (None if dt is None else g.to(dt) for g, dt in zip(grads[1:], ctx.dtypes))
        return (grads[0], *wgrads, None, None)


def layer_norm(x, gamma=None, beta=None, eps=1e-5, checkpoint=False):
    """LayerNorm over the last axis of x [..., C] (BF16, FP16 or FP32; FP32 statistics and weights).
    With ``checkpoint`` the backward pass reads an 8-bit checkpoint of x in the place of x."""
    return _LayerNorm.apply(x, gamma, beta, eps, checkpoint)


class _CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, mask, kv_lens, scale):
        Q, K, V = (_spaced(t) for t in (Q, K, V))
        mask, kv_lens = (None if t is None else t.contiguous() for t in (mask, kv_lens))
        O, LSE = tb.cross_forward(Q, K, V, mask, kv_lens, scale)
        ctx.scale = scale
        ctx.save_for_backward(Q, K, V, mask, kv_lens, O, LSE)
        return O

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        Q, K, V, mask, kv_lens, O, LSE = ctx.saved_tensors
        grads = tb.cross_backward(Q, K, V, O, LSE, _dense(dO.to(torch.bfloat16)), mask, kv_lens, ctx.scale)
        return (*grads, None, None, None)


def _spaced(t):
    """t as the kernels read it in place (channels contiguous, the other strides multiples of 8 elements and not
    zero, a 16-byte aligned start), else a contiguous copy."""
    fits = t.dim() == 4 and (t.stride(3) == 1 or t.shape[3] == 1) and t.data_ptr() % 16 == 0 and all(
        n == 1 or (s >= t.shape[3] and s % 8 == 0) for n, s in zip(t.shape[:3], t.stride()[:3]))
    return t if fits else _dense(t)


def cross_attention(Q, K, V, mask=None, kv_lens=None, scale=None):
    """Cross attention of BF16 CUDA queries Q [B, T, H, d] to encoder states K, V [B, S, Hk, d] (H a multiple of
    Hk; include/tri_cross.h): mask [B, S] False where a key is not attended, kv_lens int32 [B]. Parts of fused
    projections and transposed heads are read in place."""
    return _CrossAttention.apply(Q, K, V, mask, kv_lens, scale)


class TriangleAttentionBlock(torch.nn.Module):
    """The triangle-attention block as a module with FP32 master parameters (initialised like the
    seeded test inputs: gamma 1, beta 0, W and wb normal / sqrt(c), Wo normal / sqrt(H d)).
    ``checkpoint``: keep the input in 8 bits and recompute the activations in the backward pass."""

    def __init__(self, c: int = 128, H: int = 4, d: int = 32, node: int = tb.NODE_STARTING, eps: float = 1e-5,
                 device=None, checkpoint: bool = False):
        super().__init__()
        self.c, self.H, self.d, self.node, self.eps, self.checkpoint = c, H, d, node, eps, checkpoint
        f32 = dict(dtype=torch.float32, device=device)
        self.gamma = torch.nn.Parameter(torch.ones(c, **f32))
        self.beta = torch.nn.Parameter(torch.zeros(c, **f32))
        self.W = torch.nn.Parameter(torch.randn(4 * H * d, c, **f32) / math.sqrt(c))
        self.wb = torch.nn.Parameter(torch.randn(H, c, **f32) / math.sqrt(c))
        self.Wo = torch.nn.Parameter(torch.randn(c, H * d, **f32) / math.sqrt(H * d))

    def forward(self, z, mask=None):
        return triangle_attention_block(z, self.gamma, self.beta, self.W, self.wb, self.Wo, mask, self.H, self.d,
                                        self.node, self.eps, self.checkpoint)


class _RelativePositionBias(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, base, starts, Nq, Nk, B, two_sided, positions, key_positions):
        base = None if base is None else _dense(base)
        positions, key_positions = (None if t is None else t.contiguous() for t in (positions, key_positions))
        ctx.cfg = (starts, two_sided, table.dtype)
        ctx.save_for_backward(positions, key_positions)
        return tb.relpos_forward(table.float().contiguous(), starts, Nq, Nk, B, two_sided, base, positions, key_positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dbias):
        positions, key_positions = ctx.saved_tensors
        starts, two_sided, dtype = ctx.cfg
        dtable = None
        if ctx.needs_input_grad[0]:
            dtable = tb.relpos_backward(_dense(dbias.to(torch.bfloat16)), starts, two_sided, positions, key_positions).to(dtype)
        return (dtable, dbias if ctx.needs_input_grad[1] else None, *[None] * 7)


def relative_position_bias(table, starts, Nq, Nk=None, B=1, base=None, two_sided=True, positions=None, key_positions=None):
    """The BF16 pair bias [B, H, Nq, Nk] that triangle_attention takes: base + table[bucket(key's position - query's)].
    table [2 K, H] (one-sided: [K, H]); starts: the buckets' first distances (binding.relpos_starts makes logarithmic ones);
    base BF16 [B, H, Nq, Nk] or None; positions int32 [B, Nq] and key_positions [B, Nk] (None: 0, 1, 2, ...)."""
    return _RelativePositionBias.apply(table, base, tuple(int(s) for s in starts), Nq, Nk, B, two_sided, positions, key_positions)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, residual, eps):
        x = x.contiguous()
        g32 = None if gamma is None else gamma.float().contiguous()
        got = tb.rms_forward(x, g32, None if residual is None else residual.contiguous(), eps=eps)
        ctx.dtype = None if gamma is None else gamma.dtype
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if got.r is None else got.r, g32, got.rstd)
        return got.y if got.r is None else (got.y, got.r)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr=None):
        r, g32, rstd = ctx.saved_tensors
        if dy is None:  # (only the sum was used)
            return dr, None, dr, None
        dx, dgamma = tb.rms_backward(r, g32, rstd, dy.contiguous(), None if dr is None else dr.contiguous())
        return dx, None if dgamma is None else dgamma.to(ctx.dtype), dx if ctx.needs_input_grad[2] else None, None


def rms_norm(x, gamma=None, residual=None, eps=1e-5):
    """RMS norm over the last axis of x [..., C] (BF16, FP16 or FP32; FP32 statistics and weights): y, and with a
    residual (y, r), the norm of r = x + residual and r, which goes on past the layer."""
    return _RmsNorm.apply(x, gamma, residual, eps)


class _GatedFeedForward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, act, checkpoint):
        x = _dense(x)
        bf = [_dense(w.to(torch.bfloat16)) for w in (Wg, Wu, Wd)]
        out, *kept = (tb.ffn_forward(x, *bf, act=act), *tb.checkpoint_pack(x)) if checkpoint else (
            *tb.ffn_forward(x, *bf, act=act, keep=True), x)
        ctx.cfg = (act, checkpoint, [w.dtype for w in (Wg, Wu, Wd)])
        ctx.save_for_backward(*bf, *kept)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        act, checkpoint, dtypes = ctx.cfg
        Wg, Wu, Wd, *kept = ctx.saved_tensors
        if checkpoint:
            x = tb.checkpoint_unpack(kept)
            a, u = tb.ffn_forward(x, Wg, Wu, Wd, act=act, keep="only")
        else:
            a, u, x = kept
        return (*_ffn_gradients(ctx.needs_input_grad[:4], x, (Wg, Wu, Wd), a, u, dout, act, dtypes), None, None)


def _ffn_gradients(needs, x, weights, a, u, dout, act, dtypes):
    """The gradients of x and the three weights (None where needs says so), in the weights' masters' dtypes: from FP32 ones
    where a master is not BF16."""
    exact = torch.bfloat16 if all(d == torch.bfloat16 for d in dtypes) else torch.float32
    dx, *dw = tb.ffn_backward(x, *weights, a, u, _dense(dout.to(torch.bfloat16)), act=act, weight_dtype=exact,
                              need_dx=needs[0], need_dw=any(needs[1:]))
    return (dx, *(g.to(d) if n else None for g, d, n in zip(dw, dtypes, needs[1:])))


def _wants_gradients(*tensors):
    """Whether the call belongs to a derivative: a backward pass, or a forward-mode one, which the autograd functions refuse
    (passed by, the outputs would come without a tangent: a derivative of zero)."""
    tensors = [t for t in tensors if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        return True
    return any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def gated_feed_forward(x, Wg, Wu, Wd, act="silu", checkpoint=False):
    """The gated feed-forward block act(x Wg^T) (x Wu^T) Wd^T on BF16 rows x [..., C]: Wg, Wu [F, C] and Wd [C, F], BF16 or
    masters of another type (the forward uses their BF16 rounding); act "silu", "gelu" or "sigmoid". With ``checkpoint``
    it keeps x in 8 bits in the place of x and both projections, and its gradients are those at the checkpoint's values."""
    if not _wants_gradients(x, Wg, Wu, Wd):
        return tb.ffn_forward(_dense(x), *(_dense(w.to(torch.bfloat16)) for w in (Wg, Wu, Wd)), act=act)
    return _GatedFeedForward.apply(x, Wg, Wu, Wd, act, checkpoint)


class _FeedForwardLayer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, Wg, Wu, Wd, act, eps, checkpoint):
        x, residual = x.contiguous(), residual.contiguous()
        bf = [_dense(w.to(torch.bfloat16)) for w in (Wg, Wu, Wd)]
        g32 = gamma.float().contiguous()
        got = tb.rms_forward(x, g32, residual, eps=eps, eight_bits=checkpoint)
        out, *kept = (tb.ffn_forward(got.y, *bf, act=act), *got.y8) if checkpoint else (
            *tb.ffn_forward(got.y, *bf, act=act, keep=True), got.y)
        ctx.cfg = (act, checkpoint, gamma.dtype, [w.dtype for w in (Wg, Wu, Wd)])
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*bf, g32, got.r, got.rstd, *kept)
        return out, got.r

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dr):
        act, checkpoint, dtype, dtypes = ctx.cfg
        Wg, Wu, Wd, g32, r, rstd, *kept = ctx.saved_tensors
        if dout is None:  # (only the sum was used)
            return dr, dr, *[None] * 7
        if checkpoint:
            y = tb.checkpoint_unpack(kept)
            a, u = tb.ffn_forward(y, Wg, Wu, Wd, act=act, keep="only")
        else:
            a, u, y = kept
        needs = (any(ctx.needs_input_grad[:3]), *ctx.needs_input_grad[3:6])
        dy, *dw = _ffn_gradients(needs, y, (Wg, Wu, Wd), a, u, dout, act, dtypes)
        dx = dgamma = None
        if dy is not None:
            dx, dgamma = tb.rms_backward(r, g32, rstd, dy, None if dr is None else dr.contiguous())
            dgamma = dgamma.to(dtype)
        return (dx, dx, dgamma, *dw, None, None, None)


def feed_forward_layer(x, residual, gamma, Wg, Wu, Wd, act="silu", eps=1e-5, checkpoint=False):
    """A pre-norm feed-forward layer on BF16 rows: r = x + residual, the gated feed-forward block of r's RMS norm (weights
    gamma [C]); returns (out, r), of which the next layer takes the sum. With ``checkpoint`` the block's input is kept in 8 bits,
    written by the norm, in the place of the normalised rows and both projections, which the backward pass recomputes."""
    if not _wants_gradients(x, residual, gamma, Wg, Wu, Wd):
        got = tb.rms_forward(x.contiguous(), gamma.float().contiguous(), residual.contiguous(), eps=eps)
        return tb.ffn_forward(got.y, *(_dense(w.to(torch.bfloat16)) for w in (Wg, Wu, Wd)), act=act), got.r
    return _FeedForwardLayer.apply(x, residual, gamma, Wg, Wu, Wd, act, eps, checkpoint)


class FeedForwardLayer(torch.nn.Module):
    """The pre-norm feed-forward layer as a module with FP32 master parameters: gamma 1, the weights normal / sqrt of
    their input's width. forward(x, residual) returns (out, r)."""

    def __init__(self, C: int = 128, F: int = 512, act: str = "silu", eps: float = 1e-5, device=None, checkpoint: bool = False):
        super().__init__()
        self.act, self.eps, self.checkpoint = act, eps, checkpoint
        f32 = dict(dtype=torch.float32, device=device)
        self.gamma = torch.nn.Parameter(torch.ones(C, **f32))
        self.Wg = torch.nn.Parameter(torch.randn(F, C, **f32) / math.sqrt(C))
        self.Wu = torch.nn.Parameter(torch.randn(F, C, **f32) / math.sqrt(C))
        self.Wd = torch.nn.Parameter(torch.randn(C, F, **f32) / math.sqrt(F))

    def forward(self, x, residual):
        return feed_forward_layer(x, residual, self.gamma, self.Wg, self.Wu, self.Wd, self.act, self.eps, self.checkpoint)


def clip_grad_norm_(parameters, max_norm):
    """Clips the gradients of the parameters (those that have one) in place to the 2-norm max_norm of all of them together
    and returns their norm before, an FP32 number on the device. They are on the current device, dense and without gaps, and
    share no memory."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = [p.grad for p in parameters if p.grad is not None]
    norm = tb.clip_gradients(grads, max_norm)
    torch.autograd.graph.increment_version(grads)  # (written where autograd does not see it)
    return norm
