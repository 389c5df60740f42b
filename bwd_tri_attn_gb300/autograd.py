"""PyTorch autograd glue over the C ABI (argument marshalling only).

Every forward and backward step runs in the library's kernels through ``binding``; these classes
only keep the tensors the backward pass needs and hand gradients back in the dtypes autograd
expects. There is no CPU path: the library raises if it is missing or a call fails. Inputs and
gradients are made contiguous, and copied to a 16-byte boundary where the library wants one (a no-op
for fresh tensors); dtypes and sizes are checked by the binding. The backward passes are
differentiable once (no second derivatives).

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
"""
from __future__ import annotations

import math

import torch
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
