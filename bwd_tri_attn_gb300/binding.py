"""Thin ctypes binding of the C ABI in ``include/tri_attn.h``, ``include/tri_mul.h``,
``include/tri_module.h``, ``include/tri_norm.h``, ``include/tri_cross.h``, ``include/tri_ffn.h``,
``include/tri_rms.h``, ``include/tri_clip.h`` and ``include/tri_relpos.h``.

Argument marshalling only: PyTorch tensors supply device pointers and the
current CUDA stream; every step of the computation runs in the library's
kernels. There is no CPU fallback: if the library is missing or a call fails,
an exception is raised.
"""
from __future__ import annotations

import array
import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

from . import _build

TRI_ATTN_OK = 0
TRI_ATTN_ERR_INVALID_ARG = -1
_lock = threading.Lock()
_lib = None


NODE_STARTING, NODE_ENDING = 0, 1  # tri_attn_shape.node


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("S", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("node", ctypes.c_int)]

    def __repr__(self):
        return (f"Shape(B={self.B}, S={self.S}, N={self.N}, H={self.H}, d={self.d}, scale={self.scale}, "
                f"node={self.node})")


class TriAttnError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")
        self.code = code


_VP = ctypes.c_void_p
EXPORTS = ("tri_attn_strerror", "tri_attn_fwd", "tri_attn_bwd_workspace_size", "tri_attn_bwd_split", "tri_attn_bwd",
           "tri_attn_device_status", "tri_attn_set_timing_events", "tri_attn_bwd_static", "tri_mul_fwd",
           "tri_mul_bwd_workspace_size", "tri_mul_bwd", "tri_module_saved_size", "tri_module_bwd_workspace_size",
           "tri_module_fwd", "tri_module_bwd", "tri_norm_fwd", "tri_norm_bwd_workspace_size", "tri_norm_bwd",
           "tri_ckpt_pack", "tri_ckpt_unpack", "tri_cross_fwd_workspace_size", "tri_cross_fwd",
           "tri_cross_bwd_workspace_size", "tri_cross_bwd", "tri_ffn_fwd_workspace_size", "tri_ffn_fwd",
           "tri_ffn_bwd_workspace_size", "tri_ffn_bwd", "tri_rms_fwd", "tri_rms_bwd_workspace_size", "tri_rms_bwd",
           "tri_grad_norm", "tri_clip", "tri_relpos_fwd", "tri_relpos_bwd_workspace_size", "tri_relpos_bwd")


LAYOUT_PAIR, LAYOUT_CHANNEL_MAJOR = 0, 1  # tri_mul_shape.layout


class MulShape(ctypes.Structure):
    """tri_mul_shape: batch, residues, channels, direction (0 outgoing, 1 incoming), layout of the
    projections and their gradients (LAYOUT_PAIR [B,N,N,C] or LAYOUT_CHANNEL_MAJOR [B,C,N,N])."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int), ("incoming", ctypes.c_int),
                ("layout", ctypes.c_int)]

    def __repr__(self):
        return (f"MulShape(B={self.B}, N={self.N}, C={self.C}, incoming={self.incoming}, "
                f"layout={self.layout})")


class ModuleShape(ctypes.Structure):
    """tri_module_shape: batch, residues, pair channels, heads, head dimension, node, LayerNorm eps."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("c", ctypes.c_int), ("H", ctypes.c_int),
                ("d", ctypes.c_int), ("node", ctypes.c_int), ("eps", ctypes.c_float)]

    def __repr__(self):
        return (f"ModuleShape(B={self.B}, N={self.N}, c={self.c}, H={self.H}, d={self.d}, node={self.node}, "
                f"eps={self.eps})")


DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2  # tri_norm_shape.dtype
CKPT_GROUP = 128  # channels that share a scale in an 8-bit checkpoint
MAX_CHANNELS = 2 ** 31 - 128  # of a checkpointed row (TRI_CKPT_MAX_C; ctypes would cut a wider one to 32 bits)


class NormShape(ctypes.Structure):
    """tri_norm_shape: rows, row strides of x and dy in elements (0: C), channels, dtype, LayerNorm eps."""
    _fields_ = [("M", ctypes.c_int64), ("ldx", ctypes.c_int64), ("lddy", ctypes.c_int64), ("C", ctypes.c_int),
                ("dtype", ctypes.c_int), ("eps", ctypes.c_float)]

    def __repr__(self):
        return (f"NormShape(M={self.M}, ldx={self.ldx}, lddy={self.lddy}, C={self.C}, dtype={self.dtype}, "
                f"eps={self.eps})")


class Checkpoint(NamedTuple):
    """An activation kept in 8 bits: q8 (int8, the activation's shape) and the FP32 scales of its groups of 128
    channels ([..., (C + 127) // 128]); it stands for q8 * scale."""
    q8: torch.Tensor
    scale: torch.Tensor


class CrossShape(ctypes.Structure):
    """tri_cross_shape: batch, queries, encoder states, query heads, key heads, head dimension, scale, and the
    strides (batch, position, head; in elements) of Q, K and V."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("S", ctypes.c_int), ("H", ctypes.c_int),
                ("Hk", ctypes.c_int), ("d", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3)]

    def __repr__(self):
        return (f"CrossShape(B={self.B}, T={self.T}, S={self.S}, H={self.H}, Hk={self.Hk}, d={self.d}, "
                f"scale={self.scale}, q_stride={list(self.q_stride)}, k_stride={list(self.k_stride)}, "
                f"v_stride={list(self.v_stride)})")


ACTIVATIONS = {"silu": 0, "gelu": 1, "sigmoid": 2}  # tri_ffn_shape.act


class FfnShape(ctypes.Structure):
    """tri_ffn_shape: rows, row strides of x and dout in elements (0: C), channels, hidden features, activation,
    weight gradients in FP32 (else BF16)."""
    _fields_ = [("M", ctypes.c_int64), ("ldx", ctypes.c_int64), ("lddout", ctypes.c_int64), ("C", ctypes.c_int),
                ("F", ctypes.c_int), ("act", ctypes.c_int), ("wgrad_fp32", ctypes.c_int)]

    def __repr__(self):
        return (f"FfnShape(M={self.M}, ldx={self.ldx}, lddout={self.lddout}, C={self.C}, F={self.F}, act={self.act}, "
                f"wgrad_fp32={self.wgrad_fp32})")


class RmsShape(ctypes.Structure):
    """tri_rms_shape: rows, row strides in elements (0: C) of x or r, of the residual or dr, and of dy, channels, dtype, eps."""
    _fields_ = [("M", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldres", ctypes.c_int64), ("lddy", ctypes.c_int64),
                ("C", ctypes.c_int), ("dtype", ctypes.c_int), ("eps", ctypes.c_float)]

    def __repr__(self):
        return (f"RmsShape(M={self.M}, ldx={self.ldx}, ldres={self.ldres}, lddy={self.lddy}, C={self.C}, "
                f"dtype={self.dtype}, eps={self.eps})")


class RmsOutput(NamedTuple):
    """What rms_forward returns; what was not asked for is None."""
    y: torch.Tensor | None  # the normalised rows
    rstd: torch.Tensor      # FP32 [...]
    r: torch.Tensor | None  # x + residual
    y8: Checkpoint | None   # the normalised rows in 8 bits


CLIP_WORKSPACE_BYTES = 16384


class ClipTensor(ctypes.Structure):
    """tri_clip_tensor: a gradient, where its clipped values go, its elements and dtype."""
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int64)]


MAX_BUCKETS = 128  # of a side of the relative position bias (TRI_RELPOS_MAX_K)


class RelposShape(ctypes.Structure):
    """tri_relpos_shape: batch, heads, queries, keys, buckets of a side, whether keys ahead have buckets of their own."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Nq", ctypes.c_int), ("Nk", ctypes.c_int),
                ("K", ctypes.c_int), ("two_sided", ctypes.c_int)]

    def __repr__(self):
        return (f"RelposShape(B={self.B}, H={self.H}, Nq={self.Nq}, Nk={self.Nk}, K={self.K}, "
                f"two_sided={self.two_sided})")

    @property
    def rows(self):
        return self.K * (2 if self.two_sided else 1)


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Loads ``libtriattn.so`` (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first (__graft_entry__.build())")
        lib = ctypes.CDLL(path)
        lib.tri_attn_strerror.argtypes = [ctypes.c_int]
        lib.tri_attn_strerror.restype = ctypes.c_char_p
        lib.tri_attn_fwd.argtypes = [Shape] + [_VP] * 9
        lib.tri_attn_fwd.restype = ctypes.c_int
        lib.tri_attn_bwd_workspace_size.argtypes = [Shape]
        lib.tri_attn_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_attn_bwd_split.argtypes = [Shape, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                           ctypes.POINTER(ctypes.c_int)]
        lib.tri_attn_bwd_split.restype = ctypes.c_int
        lib.tri_attn_bwd.argtypes = [Shape] + [_VP] * 14 + [ctypes.c_size_t, _VP]
        lib.tri_attn_bwd.restype = ctypes.c_int
        lib.tri_attn_device_status.argtypes = [_VP]
        lib.tri_attn_device_status.restype = ctypes.c_int
        lib.tri_attn_bwd_static.argtypes = [Shape] + [_VP] * 14
        lib.tri_attn_bwd_static.restype = ctypes.c_int
        lib.tri_attn_set_timing_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
        lib.tri_attn_set_timing_events.restype = ctypes.c_int
        lib.tri_mul_fwd.argtypes = [MulShape] + [_VP] * 8
        lib.tri_mul_fwd.restype = ctypes.c_int
        lib.tri_mul_bwd_workspace_size.argtypes = [MulShape]
        lib.tri_mul_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_mul_bwd.argtypes = [MulShape] + [_VP] * 12 + [ctypes.c_size_t, _VP]
        lib.tri_mul_bwd.restype = ctypes.c_int
        lib.tri_module_saved_size.argtypes = [ModuleShape]
        lib.tri_module_saved_size.restype = ctypes.c_size_t
        lib.tri_module_bwd_workspace_size.argtypes = [ModuleShape]
        lib.tri_module_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_module_fwd.argtypes = [ModuleShape] + [_VP] * 9 + [ctypes.c_size_t, _VP]
        lib.tri_module_fwd.restype = ctypes.c_int
        lib.tri_module_bwd.argtypes = [ModuleShape] + [_VP] * 8 + [ctypes.c_size_t] + [_VP] * 8 + [ctypes.c_size_t, _VP]
        lib.tri_module_bwd.restype = ctypes.c_int
        lib.tri_norm_fwd.argtypes = [NormShape] + [_VP] * 9
        lib.tri_norm_fwd.restype = ctypes.c_int
        lib.tri_norm_bwd_workspace_size.argtypes = [NormShape]
        lib.tri_norm_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_norm_bwd.argtypes = [NormShape] + [_VP] * 11 + [ctypes.c_size_t, _VP]
        lib.tri_norm_bwd.restype = ctypes.c_int
        lib.tri_ckpt_pack.argtypes = [NormShape] + [_VP] * 4
        lib.tri_ckpt_pack.restype = ctypes.c_int
        lib.tri_ckpt_unpack.argtypes = [NormShape] + [_VP] * 4
        lib.tri_ckpt_unpack.restype = ctypes.c_int
        lib.tri_cross_fwd_workspace_size.argtypes = [CrossShape]
        lib.tri_cross_fwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_cross_fwd.argtypes = [CrossShape] + [_VP] * 8 + [ctypes.c_size_t, _VP]
        lib.tri_cross_fwd.restype = ctypes.c_int
        lib.tri_cross_bwd_workspace_size.argtypes = [CrossShape]
        lib.tri_cross_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_cross_bwd.argtypes = [CrossShape] + [_VP] * 12 + [ctypes.c_size_t, _VP]
        lib.tri_cross_bwd.restype = ctypes.c_int
        lib.tri_ffn_fwd_workspace_size.argtypes = [FfnShape]
        lib.tri_ffn_fwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_ffn_fwd.argtypes = [FfnShape] + [_VP] * 8 + [ctypes.c_size_t, _VP]
        lib.tri_ffn_fwd.restype = ctypes.c_int
        lib.tri_ffn_bwd_workspace_size.argtypes = [FfnShape]
        lib.tri_ffn_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_ffn_bwd.argtypes = [FfnShape] + [_VP] * 12 + [ctypes.c_size_t, _VP]
        lib.tri_ffn_bwd.restype = ctypes.c_int
        lib.tri_rms_fwd.argtypes = [RmsShape] + [_VP] * 9
        lib.tri_rms_fwd.restype = ctypes.c_int
        lib.tri_rms_bwd_workspace_size.argtypes = [RmsShape]
        lib.tri_rms_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_rms_bwd.argtypes = [RmsShape] + [_VP] * 8 + [ctypes.c_size_t, _VP]
        lib.tri_rms_bwd.restype = ctypes.c_int
        lib.tri_grad_norm.argtypes = [ctypes.c_int, _VP, _VP, _VP, ctypes.c_size_t, _VP]
        lib.tri_grad_norm.restype = ctypes.c_int
        lib.tri_clip.argtypes = [ctypes.c_int, _VP, ctypes.c_float, _VP, _VP, ctypes.c_size_t, _VP]
        lib.tri_clip.restype = ctypes.c_int
        lib.tri_relpos_fwd.argtypes = [RelposShape] + [_VP] * 7
        lib.tri_relpos_fwd.restype = ctypes.c_int
        lib.tri_relpos_bwd_workspace_size.argtypes = [RelposShape]
        lib.tri_relpos_bwd_workspace_size.restype = ctypes.c_size_t
        lib.tri_relpos_bwd.argtypes = [RelposShape] + [_VP] * 6 + [ctypes.c_size_t, _VP]
        lib.tri_relpos_bwd.restype = ctypes.c_int
        _lib = lib
    return _lib


def strerror(code: int) -> str:
    return load().tri_attn_strerror(int(code)).decode()


def shape_of(Q: torch.Tensor, scale: float | None = None, node: int = NODE_STARTING) -> Shape:
    """Shape of the attention on the pair tensor Q: [B, S, N, H, d] for the starting node (slices
    along pair axis 1), [B, N, S, H, d] for the ending node (slices along pair axis 2)."""
    B, P1, P2, H, d = (int(x) for x in Q.shape)
    S, N = (P1, P2) if node == NODE_STARTING else (P2, P1)
    return Shape(B, S, N, H, d, float(1.0 / math.sqrt(d) if scale is None else scale), int(node))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


_BF16, _F32 = torch.bfloat16, torch.float32


def _arg(t, name, dtype, numel, nullable=False):
    """Checks tensor argument `name` for what the C ABI cannot check on a bare pointer: dtype,
    contiguity and the element count the shape implies (None: any). Returns it for _ptrs, which
    checks the devices once every argument has passed these checks."""
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, the shape needs {numel}")
    return (name, t)


def _ptrs(*checked):
    """Device pointers of arguments that passed _arg: each a CUDA tensor on the current device (a
    wrong tensor raises here instead of being read or written out of bounds)."""
    out = []
    for c in checked:
        if c is None:
            out.append(None)
            continue
        name, t = c
        if not t.is_cuda or t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} must be a CUDA tensor on the current device, got {t.device}")
        out.append(ctypes.c_void_p(t.data_ptr()))
    return out


def _attn_counts(shape):
    pair = shape.B * shape.S * shape.N * shape.H * shape.d
    return pair, shape.B * shape.H * shape.N * shape.N, shape.B * shape.S * shape.N, shape.B * shape.S * shape.H * shape.N


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_device(device, *checked):
    """Raises unless every argument that passed _arg is a CUDA tensor on the current device, and returns that
    device's index (device: the first argument's get_device())."""
    for c in checked:
        if c is not None and (c[1].get_device() != device or device < 0):
            break
    else:
        if device >= 0 and device == torch.cuda.current_device():
            return device
    _ptrs(*checked)  # (names the argument)
    return device


def _raw_stream(device):
    """The raw handle of the device's current stream (as _stream, with less work on the host)."""
    return _raw_stream_of(device) if _raw_stream_of is not None else torch.cuda.current_stream().cuda_stream


def _other_stream(stream):
    """The stream that an allocating helper was given (a torch stream or a raw handle), if it is not the current one."""
    if stream is None:
        return None
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != torch.cuda.current_device():
        raise ValueError(f"stream must be one of the current device's, got {stream}")
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    current = torch.cuda.current_stream().cuda_stream
    if handle == current or (handle, current) == (1, 0):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if handle == 2:  # cudaStreamPerThread: torch can make no stream object of it, and so cannot keep its memory
        raise ValueError("the per-thread default stream cannot be given to a call that allocates")
    return torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()  # (1: cudaStreamLegacy)


def _called_on(stream, call, *args, workspace=None, **kwargs):
    """call(*args) with `stream` in the place of the caller's current one. What it allocates is that stream's memory:
    memory that the caller's stream has been given back may still be in use by what runs there. The results are not
    given out again before the caller's stream has passed whatever it does with them until they are dropped."""
    caller = torch.cuda.current_stream()
    if workspace is not None:
        kwargs["workspace"] = workspace
    with torch.cuda.stream(stream):
        out = call(*args, **kwargs)
    if workspace is not None:
        workspace.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        for r in t if isinstance(t, tuple) else (t,):
            if r is not None:
                r.record_stream(caller)
    return out


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(fn, rc):
    if rc != TRI_ATTN_OK:
        raise TriAttnError(fn, rc)


def tri_attn_fwd(shape: Shape, Q, K, V, bias, mask, O, LSE, Ores, stream=None):
    pair, nb, nm, nl = _attn_counts(shape)
    ptrs = _ptrs(_arg(Q, "Q", _BF16, pair), _arg(K, "K", _BF16, pair), _arg(V, "V", _BF16, pair),
                 _arg(bias, "bias", _BF16, nb), _arg(mask, "mask", _BF16, nm, True), _arg(O, "O", _BF16, pair),
                 _arg(LSE, "LSE", _F32, nl), _arg(Ores, "Ores", _BF16, pair, True))
    rc = load().tri_attn_fwd(shape, *ptrs, _stream(stream))
    _check("tri_attn_fwd", rc)


def tri_attn_bwd_workspace_size(shape: Shape) -> int:
    return int(load().tri_attn_bwd_workspace_size(shape))


def tri_attn_bwd_split(shape: Shape, static_entry: bool = False) -> tuple[int, int]:
    """(clusters, dBias partial slots per head) of the backward's work split on the current device."""
    nc, slots = ctypes.c_int(0), ctypes.c_int(0)
    rc = load().tri_attn_bwd_split(shape, int(bool(static_entry)), ctypes.byref(nc), ctypes.byref(slots))
    _check("tri_attn_bwd_split", rc)
    return nc.value, slots.value


def _attn_bwd_args(shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias):
    pair, nb, nm, nl = _attn_counts(shape)
    return [_arg(Q, "Q", _BF16, pair), _arg(K, "K", _BF16, pair), _arg(V, "V", _BF16, pair),
            _arg(bias, "bias", _BF16, nb), _arg(mask, "mask", _BF16, nm, True), _arg(O, "O", _BF16, pair),
            _arg(Ores, "Ores", _BF16, pair, True), _arg(LSE, "LSE", _F32, nl), _arg(dO, "dO", _BF16, pair),
            _arg(dQ, "dQ", _BF16, pair), _arg(dK, "dK", _BF16, pair), _arg(dV, "dV", _BF16, pair),
            _arg(dBias, "dBias", _BF16, nb)]


def tri_attn_bwd(shape: Shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias, workspace,
                 stream=None):
    ptrs = _ptrs(*_attn_bwd_args(shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias),
                 _arg(workspace, "workspace", None, None, True))
    rc = load().tri_attn_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_attn_bwd", rc)


def tri_attn_bwd_static(shape: Shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias, stream=None):
    """Backward pass with the library's static scratch array (no workspace argument)."""
    ptrs = _ptrs(*_attn_bwd_args(shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias))
    rc = load().tri_attn_bwd_static(shape, *ptrs, _stream(stream))
    _check("tri_attn_bwd_static", rc)


def tri_mul_fwd(shape: MulShape, Pa, Ga, Pb, Gb, A, Bm, X, stream=None):
    n = shape.B * shape.N * shape.N * shape.C
    ptrs = _ptrs(*[_arg(t, k, _BF16, n) for t, k in ((Pa, "Pa"), (Ga, "Ga"), (Pb, "Pb"), (Gb, "Gb"), (A, "A"),
                                                     (Bm, "Bm"), (X, "X"))])
    rc = load().tri_mul_fwd(shape, *ptrs, _stream(stream))
    _check("tri_mul_fwd", rc)


def tri_mul_bwd_workspace_size(shape: MulShape) -> int:
    return int(load().tri_mul_bwd_workspace_size(shape))


def tri_mul_bwd(shape: MulShape, Pa, Ga, Pb, Gb, A, Bm, dX, dPa, dGa, dPb, dGb, workspace, stream=None):
    n = shape.B * shape.N * shape.N * shape.C
    ptrs = _ptrs(*[_arg(t, k, _BF16, n) for t, k in ((Pa, "Pa"), (Ga, "Ga"), (Pb, "Pb"), (Gb, "Gb"), (A, "A"),
                                                     (Bm, "Bm"), (dX, "dX"), (dPa, "dPa"), (dGa, "dGa"),
                                                     (dPb, "dPb"), (dGb, "dGb"))],
                 _arg(workspace, "workspace", None, None, True))
    rc = load().tri_mul_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_mul_bwd", rc)


def tri_module_saved_size(shape: ModuleShape) -> int:
    return int(load().tri_module_saved_size(shape))


def tri_module_bwd_workspace_size(shape: ModuleShape) -> int:
    return int(load().tri_module_bwd_workspace_size(shape))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _module_args(shape, z, gamma, beta, W, wb, Wo, mask):
    B, N, c, hd = shape.B, shape.N, shape.c, shape.H * shape.d
    return [_arg(z, "z", _BF16, B * N * N * c), _arg(gamma, "gamma", _F32, c), _arg(beta, "beta", _F32, c),
            _arg(W, "W", _BF16, 4 * hd * c), _arg(wb, "wb", _BF16, shape.H * c), _arg(Wo, "Wo", _BF16, c * hd),
            _arg(mask, "mask", _BF16, B * N * N, True)]


def tri_module_fwd(shape: ModuleShape, z, gamma, beta, W, wb, Wo, mask, out, saved, stream=None):
    n = shape.B * shape.N * shape.N * shape.c
    ptrs = _ptrs(*_module_args(shape, z, gamma, beta, W, wb, Wo, mask), _arg(out, "out", _BF16, n),
                 _arg(saved, "saved", None, None, True))
    rc = load().tri_module_fwd(shape, *ptrs, _nbytes(saved), _stream(stream))
    _check("tri_module_fwd", rc)


def tri_module_bwd(shape: ModuleShape, z, gamma, beta, W, wb, Wo, mask, saved, dout, dz, dgamma, dbeta, dW, dwb,
                   dWo, workspace, stream=None):
    n, c, hd = shape.B * shape.N * shape.N * shape.c, shape.c, shape.H * shape.d
    p = _ptrs(*_module_args(shape, z, gamma, beta, W, wb, Wo, mask), _arg(saved, "saved", None, None, True),
              _arg(dout, "dout", _BF16, n), _arg(dz, "dz", _BF16, n), _arg(dgamma, "dgamma", _F32, c),
              _arg(dbeta, "dbeta", _F32, c), _arg(dW, "dW", _F32, 4 * hd * c), _arg(dwb, "dwb", _F32, shape.H * c),
              _arg(dWo, "dWo", _F32, c * hd), _arg(workspace, "workspace", None, None, True))
    # (z .. mask, saved | dout .. dWo, workspace)
    rc = load().tri_module_bwd(shape, *p[:8], _nbytes(saved), *p[8:16], _nbytes(workspace), _stream(stream))
    _check("tri_module_bwd", rc)


_NORM_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32}


def _norm_dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _NORM_DTYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return _NORM_DTYPES[t.dtype]


def _row_stride(t, name):
    """Elements between the rows of `t` [..., C] when its rows are contiguous and evenly spaced."""
    if t.is_contiguous():
        return t.shape[-1]
    ld, expect = None, None
    if t.shape[-1] == 1 or t.stride(-1) == 1:
        for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
            if n == 1:
                continue
            if ld is None:
                ld = s
            elif s != expect:
                ld = -1
                break
            expect = s * n
    if ld is None or ld < t.shape[-1]:
        raise ValueError(f"{name} must have contiguous, evenly spaced rows, got strides {t.stride()} for shape "
                         f"{tuple(t.shape)}")
    return ld


def _rows_arg(t, name, dtype, numel):
    """As _arg, for a tensor whose rows may be spaced apart (_row_stride has checked them)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, the shape needs {numel}")
    return (name, t)


def _channels(t, name):
    C = t.shape[-1]
    if C > MAX_CHANNELS:
        raise ValueError(f"{name} has rows of {C} channels, of which there may be {MAX_CHANNELS}")
    return C


def _norm_counts(shape):
    return shape.M * shape.C, shape.M * ((shape.C + CKPT_GROUP - 1) // CKPT_GROUP)


_TORCH_DTYPES = {v: k for k, v in _NORM_DTYPES.items()}


def _spaced_arg(t, name, dtype, shape, ld):
    """An [M, C] tensor argument with `ld` elements between its rows (0: C)."""
    if ld in (0, shape.C):
        return _arg(t, name, dtype, shape.M * shape.C)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if _row_stride(t, name) != ld or t.shape[-1] != shape.C:
        raise ValueError(f"{name}'s rows are not the {ld} elements apart that the shape gives")
    return _rows_arg(t, name, dtype, shape.M * shape.C)


def tri_norm_fwd(shape: NormShape, x, gamma, beta, y, mean, rstd, q8=None, scale=None, stream=None):
    n, ng = _norm_counts(shape)
    dt = _TORCH_DTYPES.get(shape.dtype)
    ptrs = _ptrs(_spaced_arg(x, "x", dt, shape, shape.ldx), _arg(gamma, "gamma", _F32, shape.C, True),
                 _arg(beta, "beta", _F32, shape.C, True), _arg(y, "y", dt, n), _arg(mean, "mean", _F32, shape.M),
                 _arg(rstd, "rstd", _F32, shape.M), _arg(q8, "q8", torch.int8, n, True),
                 _arg(scale, "scale", _F32, ng, True))
    rc = load().tri_norm_fwd(shape, *ptrs, _stream(stream))
    _check("tri_norm_fwd", rc)


def tri_norm_bwd_workspace_size(shape: NormShape) -> int:
    return int(load().tri_norm_bwd_workspace_size(shape))


def tri_norm_bwd(shape: NormShape, x, q8, scale, gamma, mean, rstd, dy, dx, dgamma, dbeta, workspace, stream=None):
    n, ng = _norm_counts(shape)
    dt = _TORCH_DTYPES.get(shape.dtype)
    ptrs = _ptrs(None if x is None else _spaced_arg(x, "x", dt, shape, shape.ldx),
                 _arg(q8, "q8", torch.int8, n, True), _arg(scale, "scale", _F32, ng, True),
                 _arg(gamma, "gamma", _F32, shape.C, True), _arg(mean, "mean", _F32, shape.M),
                 _arg(rstd, "rstd", _F32, shape.M), _spaced_arg(dy, "dy", dt, shape, shape.lddy),
                 _arg(dx, "dx", dt, n), _arg(dgamma, "dgamma", _F32, shape.C, True),
                 _arg(dbeta, "dbeta", _F32, shape.C, True), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_norm_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_norm_bwd", rc)


def tri_ckpt_pack(shape: NormShape, x, q8, scale, stream=None):
    n, ng = _norm_counts(shape)
    ptrs = _ptrs(_spaced_arg(x, "x", _TORCH_DTYPES.get(shape.dtype), shape, shape.ldx),
                 _arg(q8, "q8", torch.int8, n), _arg(scale, "scale", _F32, ng))
    rc = load().tri_ckpt_pack(shape, *ptrs, _stream(stream))
    _check("tri_ckpt_pack", rc)


def tri_ckpt_unpack(shape: NormShape, q8, scale, x, stream=None):
    n, ng = _norm_counts(shape)
    ptrs = _ptrs(_arg(q8, "q8", torch.int8, n), _arg(scale, "scale", _F32, ng),
                 _arg(x, "x", _TORCH_DTYPES.get(shape.dtype), n))
    rc = load().tri_ckpt_unpack(shape, *ptrs, _stream(stream))
    _check("tri_ckpt_unpack", rc)


def _strided_arg(t, name, shape, strides):
    """A BF16 [B, n, heads, d] argument with the given strides (batch, position, head)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if t.stride(3) != 1 and shape[3] != 1:
        raise ValueError(f"{name}'s last axis must be contiguous, got strides {t.stride()}")
    for n, have, given in zip(shape, t.stride(), strides):
        if n > 1 and have != given:
            raise ValueError(f"{name} has strides {t.stride()}, the shape gives {tuple(strides)}")
    return (name, t)


def _cross_args(shape, Q, K, V, mask, kv_lens):
    B, T, S, H, Hk, d = shape.B, shape.T, shape.S, shape.H, shape.Hk, shape.d
    m = None if mask is None else mask.view(torch.uint8) if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool else mask
    return [_strided_arg(Q, "Q", (B, T, H, d), shape.q_stride), _strided_arg(K, "K", (B, S, Hk, d), shape.k_stride),
            _strided_arg(V, "V", (B, S, Hk, d), shape.v_stride), _arg(m, "mask", torch.uint8, B * S, True),
            _arg(kv_lens, "kv_lens", torch.int32, B, True)]


def tri_cross_fwd_workspace_size(shape: CrossShape) -> int:
    return int(load().tri_cross_fwd_workspace_size(shape))


def tri_cross_fwd(shape: CrossShape, Q, K, V, mask, kv_lens, O, LSE, workspace, stream=None):
    rows = shape.B * shape.T * shape.H
    ptrs = _ptrs(*_cross_args(shape, Q, K, V, mask, kv_lens), _arg(O, "O", _BF16, rows * shape.d),
                 _arg(LSE, "LSE", _F32, rows), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_cross_fwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_cross_fwd", rc)


def tri_cross_bwd_workspace_size(shape: CrossShape) -> int:
    return int(load().tri_cross_bwd_workspace_size(shape))


def tri_cross_bwd(shape: CrossShape, Q, K, V, mask, kv_lens, O, LSE, dO, dQ, dK, dV, workspace, stream=None):
    rows, keys = shape.B * shape.T * shape.H, shape.B * shape.S * shape.Hk * shape.d
    ptrs = _ptrs(*_cross_args(shape, Q, K, V, mask, kv_lens), _arg(O, "O", _BF16, rows * shape.d),
                 _arg(LSE, "LSE", _F32, rows), _arg(dO, "dO", _BF16, rows * shape.d),
                 _arg(dQ, "dQ", _BF16, rows * shape.d), _arg(dK, "dK", _BF16, keys), _arg(dV, "dV", _BF16, keys),
                 _arg(workspace, "workspace", None, None, True))
    rc = load().tri_cross_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_cross_bwd", rc)


def _ffn_args(shape, x, Wg, Wu, Wd):
    n = shape.C * shape.F
    return [_spaced_arg(x, "x", _BF16, shape, shape.ldx), _arg(Wg, "Wg", _BF16, n), _arg(Wu, "Wu", _BF16, n),
            _arg(Wd, "Wd", _BF16, n)]


def tri_ffn_fwd_workspace_size(shape: FfnShape) -> int:
    return int(load().tri_ffn_fwd_workspace_size(shape))


def tri_ffn_fwd(shape: FfnShape, x, Wg, Wu, Wd, out, a, u, workspace, stream=None):
    hidden = shape.M * shape.F
    ptrs = _ptrs(*_ffn_args(shape, x, Wg, Wu, Wd), _arg(out, "out", _BF16, shape.M * shape.C, True),
                 _arg(a, "a", _BF16, hidden, True), _arg(u, "u", _BF16, hidden, True),
                 _arg(workspace, "workspace", None, None, True))
    rc = load().tri_ffn_fwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_ffn_fwd", rc)


def tri_ffn_bwd_workspace_size(shape: FfnShape) -> int:
    return int(load().tri_ffn_bwd_workspace_size(shape))


def tri_ffn_bwd(shape: FfnShape, x, Wg, Wu, Wd, a, u, dout, dx, dWg, dWu, dWd, workspace, stream=None):
    n, hidden, wd = shape.C * shape.F, shape.M * shape.F, _F32 if shape.wgrad_fp32 else _BF16
    ptrs = _ptrs(*_ffn_args(shape, x, Wg, Wu, Wd), _arg(a, "a", _BF16, hidden), _arg(u, "u", _BF16, hidden),
                 _spaced_arg(dout, "dout", _BF16, shape, shape.lddout), _arg(dx, "dx", _BF16, shape.M * shape.C, True),
                 _arg(dWg, "dWg", wd, n, True), _arg(dWu, "dWu", wd, n, True), _arg(dWd, "dWd", wd, n, True),
                 _arg(workspace, "workspace", None, None, True))
    rc = load().tri_ffn_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_ffn_bwd", rc)


def tri_rms_fwd(shape: RmsShape, x, residual, gamma, r, y, rstd, q8=None, scale=None, stream=None):
    n, ng = _norm_counts(shape)
    dt = _TORCH_DTYPES.get(shape.dtype)
    ptrs = _ptrs(_spaced_arg(x, "x", dt, shape, shape.ldx),
                 None if residual is None else _spaced_arg(residual, "residual", dt, shape, shape.ldres),
                 _arg(gamma, "gamma", _F32, shape.C, True), _arg(r, "r", dt, n, True), _arg(y, "y", dt, n, True),
                 _arg(rstd, "rstd", _F32, shape.M), _arg(q8, "q8", torch.int8, n, True), _arg(scale, "scale", _F32, ng, True))
    rc = load().tri_rms_fwd(shape, *ptrs, _stream(stream))
    _check("tri_rms_fwd", rc)


def tri_rms_bwd_workspace_size(shape: RmsShape) -> int:
    return int(load().tri_rms_bwd_workspace_size(shape))


def tri_rms_bwd(shape: RmsShape, r, gamma, rstd, dy, dr, dx, dgamma, workspace, stream=None):
    n, _ = _norm_counts(shape)
    dt = _TORCH_DTYPES.get(shape.dtype)
    ptrs = _ptrs(_spaced_arg(r, "r", dt, shape, shape.ldx), _arg(gamma, "gamma", _F32, shape.C, True),
                 _arg(rstd, "rstd", _F32, shape.M), _spaced_arg(dy, "dy", dt, shape, shape.lddy),
                 None if dr is None else _spaced_arg(dr, "dr", dt, shape, shape.ldres), _arg(dx, "dx", dt, n),
                 _arg(dgamma, "dgamma", _F32, shape.C, True), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_rms_bwd(shape, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_rms_bwd", rc)


def tri_grad_norm(tensors, norm, workspace, stream=None):
    """``tensors``: a ctypes array of ClipTensor (device pointers that the caller answers for)."""
    ptrs = _ptrs(_arg(norm, "norm", _F32, 1), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_grad_norm(len(tensors), tensors, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_grad_norm", rc)


def tri_clip(tensors, max_norm, norm, workspace, stream=None):
    """As tri_grad_norm, and the clipped gradients."""
    ptrs = _ptrs(_arg(norm, "norm", _F32, 1), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_clip(len(tensors), tensors, max_norm, *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_clip", rc)


_I32 = torch.int32


def _starts_array(shape, starts):
    """The buckets' first distances as the library reads them (from host memory)."""
    if len(starts) != shape.K or not len(starts):
        raise ValueError(f"starts has {len(starts)} buckets, the shape {shape.K}")
    starts = [int(s) for s in starts]
    if starts[0] != 0 or any(b <= a for a, b in zip(starts, starts[1:])) or starts[-1] >= 1 << 31:
        raise ValueError(f"starts must begin with 0 and rise, below 2^31, got {starts}")
    return (ctypes.c_int32 * shape.K)(*starts)


def _positions_args(shape, positions, key_positions):
    return [_arg(positions, "positions", _I32, shape.B * shape.Nq, True),
            _arg(key_positions, "key_positions", _I32, shape.B * shape.Nk, True)]


def tri_relpos_fwd(shape: RelposShape, starts, table, positions, key_positions, base, bias, stream=None):
    n = shape.B * shape.H * shape.Nq * shape.Nk
    ptrs = _ptrs(_arg(table, "table", _F32, shape.rows * shape.H), *_positions_args(shape, positions, key_positions),
                 _arg(base, "base", _BF16, n, True), _arg(bias, "bias", _BF16, n))
    rc = load().tri_relpos_fwd(shape, _starts_array(shape, starts), *ptrs, _stream(stream))
    _check("tri_relpos_fwd", rc)


def tri_relpos_bwd_workspace_size(shape: RelposShape) -> int:
    return int(load().tri_relpos_bwd_workspace_size(shape))


def tri_relpos_bwd(shape: RelposShape, starts, positions, key_positions, dbias, dtable, workspace, stream=None):
    ptrs = _ptrs(*_positions_args(shape, positions, key_positions),
                 _arg(dbias, "dbias", _BF16, shape.B * shape.H * shape.Nq * shape.Nk),
                 _arg(dtable, "dtable", _F32, shape.rows * shape.H), _arg(workspace, "workspace", None, None, True))
    rc = load().tri_relpos_bwd(shape, _starts_array(shape, starts), *ptrs, _nbytes(workspace), _stream(stream))
    _check("tri_relpos_bwd", rc)


def tri_attn_device_status(stream=None) -> int:
    return int(load().tri_attn_device_status(_stream(stream)))


_event_array = None  # keeps the pointer array alive while instrumentation is on


def tri_attn_set_timing_events(events) -> None:
    """Per-kernel timing: ``events`` is a list of recorded torch.cuda.Event (or None to switch off)."""
    global _event_array
    if not events:
        _event_array = None
        _check("tri_attn_set_timing_events", load().tri_attn_set_timing_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _event_array = arr
    _check("tri_attn_set_timing_events", load().tri_attn_set_timing_events(arr, len(events)))


# ----------------------------------------------------------------------------
# Allocating conveniences (outputs are fresh torch tensors on Q's device; those of a call that is given a
# stream belong to that stream).
# ----------------------------------------------------------------------------

def forward(Q, K, V, bias, mask=None, scale=None, residual=True, stream=None, node=NODE_STARTING):
    """Returns (O, LSE, Ores); Ores is None when ``residual`` is False. O and Ores have Q's
    layout; LSE is [B, S, H, N] in terms of the attention's slices and positions."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, forward, Q, K, V, bias, mask, scale, residual, node=node)
    shape = shape_of(Q, scale, node)
    B, S, N, H = shape.B, shape.S, shape.N, shape.H
    O = torch.empty_like(Q)
    LSE = torch.empty((B, S, H, N), dtype=torch.float32, device=Q.device)
    Ores = torch.empty_like(Q) if residual else None
    tri_attn_fwd(shape, Q, K, V, bias, mask, O, LSE, Ores, stream)
    return O, LSE, Ores


def workspace_for(shape: Shape, device) -> torch.Tensor:
    n = tri_attn_bwd_workspace_size(shape)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def backward(Q, K, V, bias, mask, O, Ores, LSE, dO, scale=None, workspace=None, stream=None,
             node=NODE_STARTING):
    """Returns (dQ, dK, dV, dBias)."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, backward, Q, K, V, bias, mask, O, Ores, LSE, dO, scale, workspace=workspace, node=node)
    shape = shape_of(Q, scale, node)
    if workspace is None:
        workspace = workspace_for(shape, Q.device)
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    dBias = torch.empty_like(bias)
    tri_attn_bwd(shape, Q, K, V, bias, mask, O, Ores, LSE, dO, dQ, dK, dV, dBias, workspace, stream)
    return dQ, dK, dV, dBias


def mul_shape_of(Pa: torch.Tensor, incoming: bool = False, layout: int = LAYOUT_PAIR) -> MulShape:
    """Shape of the triangle multiplicative update on projections [B, N, N, C] (pair layout) or
    [B, C, N, N] (channel-major)."""
    if layout == LAYOUT_PAIR:
        B, N, N2, C = (int(x) for x in Pa.shape)
    else:
        B, C, N, N2 = (int(x) for x in Pa.shape)
    if N2 != N:
        raise ValueError(f"projection must be square in its two position axes, got {tuple(Pa.shape)}")
    return MulShape(B, N, C, int(bool(incoming)), int(layout))


def mul_forward(Pa, Ga, Pb, Gb, incoming=False, layout=LAYOUT_PAIR, stream=None):
    """Returns (X, A, Bm): X [B, C, N, N] channel-major, and the gated operands A, Bm
    [B, C, N, N] that mul_backward reads."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, mul_forward, Pa, Ga, Pb, Gb, incoming, layout)
    shape = mul_shape_of(Pa, incoming, layout)
    B, N, C = shape.B, shape.N, shape.C
    A, Bm, X = (torch.empty((B, C, N, N), dtype=torch.bfloat16, device=Pa.device) for _ in range(3))
    tri_mul_fwd(shape, Pa, Ga, Pb, Gb, A, Bm, X, stream)
    return X, A, Bm


def mul_backward(Pa, Ga, Pb, Gb, A, Bm, dX, incoming=False, layout=LAYOUT_PAIR, workspace=None, stream=None):
    """Returns (dPa, dGa, dPb, dGb) in the projections' layout; dX is channel-major."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, mul_backward, Pa, Ga, Pb, Gb, A, Bm, dX, incoming, layout, workspace=workspace)
    shape = mul_shape_of(Pa, incoming, layout)
    if workspace is None:
        workspace = torch.empty(max(tri_mul_bwd_workspace_size(shape), 16), dtype=torch.uint8, device=Pa.device)
    outs = [torch.empty_like(Pa) for _ in range(4)]
    tri_mul_bwd(shape, Pa, Ga, Pb, Gb, A, Bm, dX, *outs, workspace, stream)
    return tuple(outs)


def module_shape_of(z: torch.Tensor, H: int, d: int, node: int = NODE_STARTING, eps: float = 1e-5) -> ModuleShape:
    """Shape of the triangle-attention block on the pair representation z [B, N, N, c]."""
    B, N, N2, c = (int(x) for x in z.shape)
    if N2 != N:
        raise ValueError(f"pair representation must be square, got {tuple(z.shape)}")
    return ModuleShape(B, N, c, int(H), int(d), int(node), float(eps))


def module_forward(z, gamma, beta, W, wb, Wo, mask, H, d, node=NODE_STARTING, eps=1e-5, stream=None):
    """Returns (out, saved): out [B, N, N, c] and the activations module_backward reads."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, module_forward, z, gamma, beta, W, wb, Wo, mask, H, d, node, eps)
    shape = module_shape_of(z, H, d, node, eps)
    saved = torch.empty(max(tri_module_saved_size(shape), 16), dtype=torch.uint8, device=z.device)
    out = torch.empty_like(z)
    tri_module_fwd(shape, z, gamma, beta, W, wb, Wo, mask, out, saved, stream)
    return out, saved


def module_backward(z, gamma, beta, W, wb, Wo, mask, saved, dout, H, d, node=NODE_STARTING, eps=1e-5,
                    workspace=None, stream=None):
    """Returns (dz, dgamma, dbeta, dW, dwb, dWo); the weight gradients are FP32."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, module_backward, z, gamma, beta, W, wb, Wo, mask, saved, dout, H, d, node, eps, workspace=workspace)
    shape = module_shape_of(z, H, d, node, eps)
    if workspace is None:
        workspace = torch.empty(max(tri_module_bwd_workspace_size(shape), 16), dtype=torch.uint8, device=z.device)
    dz = torch.empty_like(z)
    f32 = dict(dtype=torch.float32, device=z.device)
    dgamma, dbeta = torch.empty(gamma.shape, **f32), torch.empty(beta.shape, **f32)
    dW, dwb, dWo = torch.empty(W.shape, **f32), torch.empty(wb.shape, **f32), torch.empty(Wo.shape, **f32)
    tri_module_bwd(shape, z, gamma, beta, W, wb, Wo, mask, saved, dout, dz, dgamma, dbeta, dW, dwb, dWo, workspace,
                   stream)
    return dz, dgamma, dbeta, dW, dwb, dWo


def norm_shape_of(x: torch.Tensor, eps: float = 1e-5, dy: torch.Tensor | None = None) -> NormShape:
    """Shape of LayerNorm over the last axis of x [..., C] (and of the row strides of x and dy)."""
    dtype = _norm_dtype(x, "x")
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"x must have at least one row and one channel, got shape {tuple(x.shape)}")
    C = _channels(x, "x")
    return NormShape(x.numel() // C, _row_stride(x, "x"), C if dy is None else _row_stride(dy, "dy"), C, dtype,
                     float(eps))


def _dense_like(x):
    """An empty tensor of x's shape and dtype without gaps (empty_like is the cheapest call for it, but keeps the
    order of a strided tensor's axes)."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _empty_checkpoint(x):
    *rows, C = x.shape
    return Checkpoint(torch.empty(x.shape, dtype=torch.int8, device=x.device),
                      torch.empty((*rows, (C + CKPT_GROUP - 1) // CKPT_GROUP), dtype=_F32, device=x.device))


def norm_forward(x, gamma=None, beta=None, eps=1e-5, checkpoint=False, stream=None):
    """LayerNorm over the last axis of x [..., C]: returns (y, mean, rstd), y in x's dtype and the FP32 statistics
    [...]; with ``checkpoint`` also the 8-bit checkpoint of x, written in the same pass."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, norm_forward, x, gamma, beta, eps, checkpoint)
    shape = norm_shape_of(x, eps)
    device = _on_device(x.get_device(), ("x", x), _arg(gamma, "gamma", _F32, shape.C, True),
                        _arg(beta, "beta", _F32, shape.C, True))
    rows = x.shape[:-1]
    y, mean, rstd = _dense_like(x), torch.empty(rows, dtype=_F32, device=x.device), torch.empty(rows, dtype=_F32, device=x.device)
    kept = _empty_checkpoint(x) if checkpoint else None
    q8, scale = (kept.q8.data_ptr(), kept.scale.data_ptr()) if checkpoint else (None, None)
    rc = load().tri_norm_fwd(shape, x.data_ptr(), _ptr(gamma), _ptr(beta), y.data_ptr(), mean.data_ptr(),
                             rstd.data_ptr(), q8, scale, _raw_stream(device))
    _check("tri_norm_fwd", rc)
    return (y, mean, rstd, kept) if checkpoint else (y, mean, rstd)


def norm_backward(x, gamma, mean, rstd, dy, workspace=None, stream=None):
    """Returns (dx, dgamma, dbeta): dx in dy's dtype, the weight gradients FP32 (None when gamma is None, the
    LayerNorm without weights). ``x`` is the forward's input or its ``Checkpoint``; mean and rstd are the forward's."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, norm_backward, x, gamma, mean, rstd, dy, workspace=workspace)
    dtype = _norm_dtype(dy, "dy")
    kept = x if isinstance(x, tuple) else None
    like = kept[0] if kept is not None else x
    if not isinstance(like, torch.Tensor) or like.shape != dy.shape:
        raise ValueError(f"dy {tuple(dy.shape)} must have x's shape")
    n = dy.numel()
    if dy.dim() < 1 or n == 0:
        raise ValueError(f"dy must have at least one row and one channel, got shape {tuple(dy.shape)}")
    C = _channels(dy, "dy")
    M = n // C
    shape = NormShape(M, C if kept is not None else _row_stride(x, "x"), _row_stride(dy, "dy"), C, dtype, 0.0)
    if kept is not None:
        given = [_arg(kept[0], "q8", torch.int8, n), _arg(kept[1], "scale", _F32, _norm_counts(shape)[1])]
    else:
        given = [_rows_arg(x, "x", dy.dtype, n)]
    device = _on_device(dy.get_device(), *given, _arg(gamma, "gamma", _F32, C, True), _arg(mean, "mean", _F32, M),
                        _arg(rstd, "rstd", _F32, M), ("dy", dy), _arg(workspace, "workspace", None, None, True))
    dx = _dense_like(dy)
    dgamma = dbeta = None
    if gamma is not None:
        dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
        if workspace is None:
            workspace = _workspace(tri_norm_bwd_workspace_size(shape), dy)
    xp, q8, scale = (None, kept[0].data_ptr(), kept[1].data_ptr()) if kept is not None else (x.data_ptr(), None, None)
    rc = load().tri_norm_bwd(shape, xp, q8, scale, _ptr(gamma), mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(),
                             dx.data_ptr(), _ptr(dgamma), _ptr(dbeta), _ptr(workspace), _nbytes(workspace),
                             _raw_stream(device))
    _check("tri_norm_bwd", rc)
    return dx, dgamma, dbeta


def checkpoint_pack(x, stream=None) -> Checkpoint:
    """x [..., C] kept in 8 bits: int8 values and one FP32 scale for every 128 channels of a row."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, checkpoint_pack, x)
    shape = norm_shape_of(x)
    device = _on_device(x.get_device(), ("x", x))
    kept = _empty_checkpoint(x)
    rc = load().tri_ckpt_pack(shape, x.data_ptr(), kept.q8.data_ptr(), kept.scale.data_ptr(),
                              _raw_stream(device))
    _check("tri_ckpt_pack", rc)
    return kept


def checkpoint_unpack(kept, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for, rounded once to ``dtype``."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, checkpoint_unpack, kept, dtype)
    q8, scale = kept
    x = torch.empty(q8.shape, dtype=dtype, device=q8.device)
    shape = norm_shape_of(x)
    n, ng = _norm_counts(shape)
    device = _on_device(x.get_device(), _arg(q8, "q8", torch.int8, n), _arg(scale, "scale", _F32, ng))
    rc = load().tri_ckpt_unpack(shape, q8.data_ptr(), scale.data_ptr(), x.data_ptr(), _raw_stream(device))
    _check("tri_ckpt_unpack", rc)
    return x


def cross_shape_of(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: float | None = None) -> CrossShape:
    """Shape of the cross attention of Q [B, T, H, d] to K, V [B, S, Hk, d], with their strides."""
    for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if t.dim() != 4:
            raise ValueError(f"{name} must have four axes (batch, position, head, channel), got shape {tuple(t.shape)}")
    B, T, H, d = Q.shape
    _, S, Hk, _ = K.shape
    if max(B, T, S, H, Hk, d) >= 1 << 31:  # (ctypes would cut it to 32 bits)
        raise ValueError(f"an axis is too long: Q has shape {tuple(Q.shape)}, K {tuple(K.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 0.0
    return CrossShape(B, T, S, H, Hk, d, scale, Q.stride()[:3], K.stride()[:3], V.stride()[:3])


def _workspace(nbytes, like):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


def _cross_checked(Q, K, V, mask, kv_lens, scale, *more):
    """The call's shape and its device, with every argument checked (more: arguments that have passed _arg)."""
    shape = cross_shape_of(Q, K, V, scale)
    kv = K.shape
    if not (Q.dtype is _BF16 and K.dtype is _BF16 and V.dtype is _BF16 and V.shape == kv and kv[0] == shape.B
            and kv[3] == shape.d and Q.stride(3) == K.stride(3) == V.stride(3) == 1 and mask is None and kv_lens is None):
        more = (*_cross_args(shape, Q, K, V, mask, kv_lens), *more)  # (names what is wrong)
    return shape, _on_device(Q.get_device(), ("Q", Q), ("K", K), ("V", V), *more)


def cross_forward(Q, K, V, mask=None, kv_lens=None, scale=None, workspace=None, stream=None):
    """Cross attention of the queries Q [B, T, H, d] to the encoder states K, V [B, S, Hk, d] (BF16; heads, positions
    and batches may be spaced apart). mask: bool or uint8 [B, S], False where a key is not to be attended; kv_lens:
    int32 [B]. Returns (O, LSE): O [B, T, H, d] and the FP32 log-sum-exp [B, H, T] that cross_backward reads."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, cross_forward, Q, K, V, mask, kv_lens, scale, workspace=workspace)
    shape, device = _cross_checked(Q, K, V, mask, kv_lens, scale, _arg(workspace, "workspace", None, None, True))
    B, T, H, _ = Q.shape
    O, LSE = _dense_like(Q), torch.empty((B, H, T), dtype=_F32, device=Q.device)
    if workspace is None:
        workspace = _workspace(tri_cross_fwd_workspace_size(shape), Q)
    rc = load().tri_cross_fwd(shape, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _ptr(mask), _ptr(kv_lens),
                              O.data_ptr(), LSE.data_ptr(), _ptr(workspace), _nbytes(workspace),
                              _raw_stream(device))
    _check("tri_cross_fwd", rc)
    return O, LSE


def cross_backward(Q, K, V, O, LSE, dO, mask=None, kv_lens=None, scale=None, workspace=None, stream=None):
    """Returns (dQ, dK, dV), without gaps, for the gradient dO of cross_forward's O."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, cross_backward, Q, K, V, O, LSE, dO, mask, kv_lens, scale, workspace=workspace)
    n = Q.numel() if isinstance(Q, torch.Tensor) else None
    rows = n // Q.shape[-1] if n else None
    shape, device = _cross_checked(Q, K, V, mask, kv_lens, scale, _arg(O, "O", _BF16, n), _arg(LSE, "LSE", _F32, rows),
                                   _arg(dO, "dO", _BF16, n), _arg(workspace, "workspace", None, None, True))
    dQ, dK, dV = _dense_like(Q), _dense_like(K), _dense_like(V)
    if workspace is None:
        workspace = _workspace(tri_cross_bwd_workspace_size(shape), Q)
    rc = load().tri_cross_bwd(shape, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _ptr(mask), _ptr(kv_lens),
                              O.data_ptr(), LSE.data_ptr(), dO.data_ptr(), dQ.data_ptr(), dK.data_ptr(),
                              dV.data_ptr(), _ptr(workspace), _nbytes(workspace), _raw_stream(device))
    _check("tri_cross_bwd", rc)
    return dQ, dK, dV


def ffn_shape_of(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, act: str = "silu",
                 dout: torch.Tensor | None = None, wgrad_fp32: bool = False) -> FfnShape:
    """Shape of the gated feed-forward block on the last axis of x [..., C] with Wg, Wu [F, C] and Wd [C, F]."""
    for t, name in ((x, "x"), (Wg, "Wg"), (Wu, "Wu"), (Wd, "Wd"), *(() if dout is None else ((dout, "dout"),))):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if t.dtype != _BF16:
            raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"x must have at least one row and one channel, got shape {tuple(x.shape)}")
    C = x.shape[-1]
    if Wg.dim() != 2 or Wg.shape[1] != C:
        raise ValueError(f"Wg must have shape [F, {C}], got {tuple(Wg.shape)}")
    F = Wg.shape[0]
    if Wu.shape != (F, C):
        raise ValueError(f"Wu must have shape {(F, C)}, got {tuple(Wu.shape)}")
    if Wd.shape != (C, F):
        raise ValueError(f"Wd must have shape {(C, F)}, got {tuple(Wd.shape)}")
    if max(C, F) >= 1 << 31:  # (ctypes would cut it to 32 bits)
        raise ValueError(f"an axis is too long: Wg has shape {tuple(Wg.shape)}")
    if dout is not None and dout.shape != x.shape:
        raise ValueError(f"dout {tuple(dout.shape)} must have x's shape {tuple(x.shape)}")
    return FfnShape(x.numel() // C, _row_stride(x, "x"), C if dout is None else _row_stride(dout, "dout"), C, F,
                    ACTIVATIONS[act], int(wgrad_fp32))


def _weights_args(Wg, Wu, Wd):
    return [_arg(Wg, "Wg", _BF16, None), _arg(Wu, "Wu", _BF16, None), _arg(Wd, "Wd", _BF16, None)]


def ffn_forward(x, Wg, Wu, Wd, act="silu", keep=False, workspace=None, stream=None):
    """The gated feed-forward block act(x Wg^T) (x Wu^T) Wd^T on x [..., C] with Wg, Wu [F, C] and Wd [C, F] (BF16; rows
    of x may be spaced apart); act: "silu", "gelu" or "sigmoid". Returns out [..., C], with ``keep`` (out, a, u): also
    the two projections [..., F], which ffn_backward reads; keep="only": (a, u) alone."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, ffn_forward, x, Wg, Wu, Wd, act, keep, workspace=workspace)
    if keep not in (False, True, "only"):
        raise ValueError(f"keep must be False, True or \"only\", got {keep!r}")
    shape = ffn_shape_of(x, Wg, Wu, Wd, act)
    device = _on_device(x.get_device(), ("x", x), *_weights_args(Wg, Wu, Wd), _arg(workspace, "workspace", None, None, True))
    out = None if keep == "only" else _dense_like(x)
    a = u = None
    if keep:
        a, u = (torch.empty((*x.shape[:-1], shape.F), dtype=_BF16, device=x.device) for _ in range(2))
    if workspace is None:
        workspace = _workspace(tri_ffn_fwd_workspace_size(shape), x)
    rc = load().tri_ffn_fwd(shape, x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), _ptr(out), _ptr(a),
                            _ptr(u), _ptr(workspace), _nbytes(workspace), _raw_stream(device))
    _check("tri_ffn_fwd", rc)
    return (a, u) if out is None else (out, a, u) if keep else out


def ffn_backward(x, Wg, Wu, Wd, a, u, dout, act="silu", weight_dtype=_BF16, need_dx=True, need_dw=True, workspace=None,
                 stream=None):
    """Returns (dx, dWg, dWu, dWd) for the gradient dout of ffn_forward's out; a and u are what it kept. The weight
    gradients are BF16 or FP32 (``weight_dtype``); what is not needed is None."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, ffn_backward, x, Wg, Wu, Wd, a, u, dout, act, weight_dtype, need_dx, need_dw,
                          workspace=workspace)
    if weight_dtype not in (_BF16, _F32):
        raise TypeError(f"weight_dtype must be {_BF16} or {_F32}, got {weight_dtype}")
    if not (need_dx or need_dw):
        raise ValueError("no gradient is asked for")
    shape = ffn_shape_of(x, Wg, Wu, Wd, act, dout, weight_dtype == _F32)
    hidden = shape.M * shape.F
    device = _on_device(x.get_device(), ("x", x), *_weights_args(Wg, Wu, Wd), _arg(a, "a", _BF16, hidden),
                        _arg(u, "u", _BF16, hidden), ("dout", dout), _arg(workspace, "workspace", None, None, True))
    dx = _dense_like(x) if need_dx else None
    dWg, dWu, dWd = (torch.empty(w.shape, dtype=weight_dtype, device=w.device) if need_dw else None for w in (Wg, Wu, Wd))
    if workspace is None:
        workspace = _workspace(tri_ffn_bwd_workspace_size(shape), x)
    rc = load().tri_ffn_bwd(shape, x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), a.data_ptr(), u.data_ptr(),
                            dout.data_ptr(), _ptr(dx), _ptr(dWg), _ptr(dWu), _ptr(dWd), _ptr(workspace),
                            _nbytes(workspace), _raw_stream(device))
    _check("tri_ffn_bwd", rc)
    return dx, dWg, dWu, dWd


def rms_shape_of(x: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-5,
                 dy: torch.Tensor | None = None) -> RmsShape:
    """Shape of the RMS norm over the last axis of x [..., C] (r in the backward pass) and the row strides of it, of the
    residual (dr) and of dy."""
    dtype = _norm_dtype(x, "x")
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"x must have at least one row and one channel, got shape {tuple(x.shape)}")
    C = _channels(x, "x")
    for t, name in ((residual, "residual"), (dy, "dy")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if t.shape != x.shape:
            raise ValueError(f"{name} {tuple(t.shape)} must have x's shape {tuple(x.shape)}")
        if t.dtype != x.dtype:
            raise TypeError(f"{name} must be {x.dtype}, got {t.dtype}")
    return RmsShape(x.numel() // C, _row_stride(x, "x"), C if residual is None else _row_stride(residual, "residual"),
                    C if dy is None else _row_stride(dy, "dy"), C, dtype, float(eps))


def rms_forward(x, gamma=None, residual=None, eps=1e-5, eight_bits=False, stream=None) -> RmsOutput:
    """RMS norm over the last axis of r = x + residual (of x without a residual), x [..., C] in BF16, FP16 or FP32: returns
    RmsOutput(y, rstd, r, y8). eight_bits: also y8, y as a ``Checkpoint`` (checkpoint_unpack reads it); "only": y8 in the
    place of y. r is None without a residual."""
    if (other := _other_stream(stream)) is not None:
        return RmsOutput(*_called_on(other, rms_forward, x, gamma, residual, eps, eight_bits))
    if eight_bits not in (False, True, "only"):
        raise ValueError(f"eight_bits must be False, True or \"only\", got {eight_bits!r}")
    shape = rms_shape_of(x, residual, eps)
    device = _on_device(x.get_device(), ("x", x), None if residual is None else ("residual", residual),
                        _arg(gamma, "gamma", _F32, shape.C, True))
    r = None if residual is None else _dense_like(x)
    y = None if eight_bits == "only" else _dense_like(x)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=x.device)
    y8 = _empty_checkpoint(x) if eight_bits else None
    q8, scale = (y8.q8.data_ptr(), y8.scale.data_ptr()) if eight_bits else (None, None)
    rc = load().tri_rms_fwd(shape, x.data_ptr(), _ptr(residual), _ptr(gamma), _ptr(r), _ptr(y), rstd.data_ptr(), q8, scale,
                            _raw_stream(device))
    _check("tri_rms_fwd", rc)
    return RmsOutput(y, rstd, r, y8)


def rms_backward(r, gamma, rstd, dy, dr=None, workspace=None, stream=None):
    """Returns (dx, dgamma): dx, the gradient of x and of the residual alike, and dgamma in FP32 (None when gamma is None).
    r and rstd are the forward's (r: x where there was no residual); dr is the gradient that reaches r past the norm."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, rms_backward, r, gamma, rstd, dy, dr, workspace=workspace)
    shape = rms_shape_of(r, dr, 0.0, dy)
    device = _on_device(r.get_device(), ("r", r), ("dy", dy), None if dr is None else ("dr", dr),
                        _arg(gamma, "gamma", _F32, shape.C, True), _arg(rstd, "rstd", _F32, shape.M),
                        _arg(workspace, "workspace", None, None, True))
    dx = _dense_like(dy)
    dgamma = None
    if gamma is not None:
        dgamma = torch.empty_like(gamma)
        if workspace is None:
            workspace = _workspace(tri_rms_bwd_workspace_size(shape), dy)
    rc = load().tri_rms_bwd(shape, r.data_ptr(), _ptr(gamma), rstd.data_ptr(), dy.data_ptr(), _ptr(dr), dx.data_ptr(),
                            _ptr(dgamma), _ptr(workspace), _nbytes(workspace), _raw_stream(device))
    _check("tri_rms_bwd", rc)
    return dx, dgamma


def _gapless(t):
    """Whether a tensor's elements fill its memory, in whatever order of its axes."""
    if t.is_contiguous():  # (without elements, too)
        return True
    want = 1
    for stride, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n != 1):
        if stride != want:
            return False
        want *= n
    return True


def _same_order(g, t):
    """Whether a value of g and its product, in t, are equally far from the tensors' first elements."""
    return (g.is_contiguous() and t.is_contiguous()) or (g.shape == t.shape and g.stride() == t.stride())


def _clip_array(grads, out, written):
    """The gradients' descriptions for the library (as ClipTensor's fields one behind another), their number and the
    device's index: every tensor checked, none twice among those that are written."""
    device = torch.cuda.current_device()
    try:
        types = [g.dtype for g in grads]
        codes = [_NORM_DTYPES[t] for t in types]
        sizes = [g.numel() for g in grads]
        at = [g.data_ptr() for g in grads]
        plain = all([g.is_contiguous() for g in grads])
        fine = all([g.get_device() == device for g in grads]) and (plain or all(map(_gapless, grads)))
        to = at
        if out is not None:
            to = [t.data_ptr() for t in out]
            fine = (fine and [t.dtype for t in out] == types and [t.numel() for t in out] == sizes
                    and all([t.get_device() == device for t in out])
                    and ((plain and all([t.is_contiguous() for t in out])) or all(map(_same_order, grads, out))))
    except (AttributeError, KeyError):
        fine = False
    if not fine:
        _clip_refusal(device, grads, out)
    if 0 in sizes:
        some = [i for i, n in enumerate(sizes) if n]
        codes, sizes, at, to = ([v[i] for i in some] for v in (codes, sizes, at, to))
    n = len(at)
    if written and len(set(to)) != n:
        raise ValueError("a tensor stands twice among the gradients that are written")
    rows = array.array("q", bytes(32 * n))
    for k, v in enumerate((at, to, sizes, codes)):
        rows[k::4] = array.array("q", v)
    return rows, n, device


def _clip_refusal(device, grads, out):
    """Names what is wrong with one of the tensors."""
    for i, g in enumerate(grads):
        _norm_dtype(g, f"gradient {i}")
        for t, name in ((g, f"gradient {i}"), *(() if out is None else ((out[i], f"out {i}"),))):
            if not isinstance(t, torch.Tensor) or t.dtype != g.dtype or t.numel() != g.numel():
                raise ValueError(f"{name} must be a tensor of gradient {i}'s size and type")
            if not _gapless(t):
                raise ValueError(f"{name} must be contiguous, in whatever order of its axes")
            if t.get_device() != device:
                raise ValueError(f"{name} must be a CUDA tensor on the current device, got {t.device}")
        if out is not None and not _same_order(g, out[i]):
            raise ValueError(f"out {i} must have gradient {i}'s shape and strides, {tuple(g.shape)} and {g.stride()}, "
                             f"got {tuple(out[i].shape)} and {out[i].stride()}")
    raise ValueError("the gradients' tensors do not fit together")


def _clip(call, grads, out, workspace, *more, written=True):
    grads = list(grads)
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
    rows, count, device = _clip_array(grads, out, written)
    norm = torch.empty((), dtype=_F32, device=torch.device("cuda", device))
    if workspace is None:
        workspace = torch.empty(CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=norm.device)
    _on_device(device, _arg(workspace, "workspace", None, None))
    rc = getattr(load(), call)(count, rows.buffer_info()[0], *more, norm.data_ptr(), workspace.data_ptr(), _nbytes(workspace),
                               _raw_stream(device))
    if rc == TRI_ATTN_ERR_INVALID_ARG:  # (the rest is checked)
        raise ValueError("a tensor that is written shares memory with another one")
    _check(call, rc)
    return norm


def gradient_norm(grads, workspace=None, stream=None) -> torch.Tensor:
    """The 2-norm of all elements of the gradients (BF16, FP16 and FP32 tensors of any number and shapes, without gaps in whatever
    order of their axes; one that is named twice counts twice): an FP32 number on the device."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, gradient_norm, grads, workspace=workspace)
    return _clip("tri_grad_norm", grads, None, workspace, written=False)


def clip_gradients(grads, max_norm, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Multiplies the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors ``out``, and returns
    their norm before, an FP32 number on the device. No tensor that is written shares memory with another one; one that is
    transposed or permuted has an ``out`` of the same strides."""
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, clip_gradients, grads, max_norm, out, workspace=workspace)
    return _clip("tri_clip", grads, out, workspace, max_norm)


def relpos_starts(buckets: int, max_distance: int, two_sided: bool = True) -> tuple[int, ...]:
    """The first distances of logarithmic buckets: of ``buckets`` in all (half of them on each side if two-sided, K on a
    side) the first e = (K + 1) // 2 of a side hold one distance each, the others equal steps of the logarithm up to
    max_distance: bucket e + k holds the distances n with (n / e)^(K - e) >= (max_distance / e)^k (in whole numbers,
    so that no rounding moves a border; at least one distance a bucket)."""
    K = buckets // 2 if two_sided else buckets
    if K < 1 or (two_sided and buckets % 2):
        raise ValueError(f"there must be at least one bucket on a side, and as many on both: got {buckets}")
    if max_distance < K:
        raise ValueError(f"max_distance must be at least the {K} buckets of a side, got {max_distance}")
    e = (K + 1) // 2
    m, starts = K - e, list(range(e))
    for k in range(m):
        low, high = starts[-1] + 1 if starts else 0, max(max_distance, starts[-1] + 1)
        while low < high:
            mid = (low + high) // 2
            if mid ** m * e ** k >= max_distance ** k * e ** m:
                high = mid
            else:
                low = mid + 1
        starts.append(low)
    return tuple(starts)


def _positions_of(shape, positions, key_positions):
    if positions is None and key_positions is not None:
        raise ValueError("key_positions come with positions")
    if positions is not None and key_positions is None:
        if shape.Nq != shape.Nk:
            raise ValueError(f"{shape.Nk} keys need positions of their own, there are {shape.Nq} queries")
        key_positions = positions
    for t, name, n in ((positions, "positions", shape.Nq), (key_positions, "key_positions", shape.Nk)):
        if isinstance(t, torch.Tensor) and t.shape != (shape.B, n):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {(shape.B, n)}")
    return positions, key_positions


def _axes(*axes):
    if max(axes) >= 1 << 31:  # (ctypes would cut it to 32 bits)
        raise ValueError(f"an axis is too long: {axes}")


def relpos_forward(table, starts, Nq, Nk=None, B=1, two_sided=True, base=None, positions=None, key_positions=None,
                   stream=None) -> torch.Tensor:
    """The pair bias [B, H, Nq, Nk] (BF16) base + table[bucket(key's position - query's)]: table FP32 [rows, H], 2 K rows
    for K two-sided buckets or K; ``starts``: the buckets' first distances (relpos_starts makes logarithmic ones); base BF16
    [B, H, Nq, Nk] or None; positions int32 [B, Nq], key_positions [B, Nk] (None: 0, 1, 2, ...; the queries')."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, relpos_forward, table, starts, Nq, Nk, B, two_sided, base, positions, key_positions)
    if not isinstance(table, torch.Tensor):
        raise TypeError(f"table must be a torch.Tensor, got {type(table).__name__}")
    Nk = Nq if Nk is None else Nk
    K = len(starts)
    if table.dim() != 2 or table.shape[0] != K * (2 if two_sided else 1):
        raise ValueError(f"table must have shape [{K * (2 if two_sided else 1)}, H], got {tuple(table.shape)}")
    H = table.shape[1]
    _axes(B, H, Nq, Nk)
    shape = RelposShape(B, H, Nq, Nk, K, int(bool(two_sided)))
    if isinstance(base, torch.Tensor) and base.shape != (B, H, Nq, Nk):
        raise ValueError(f"base has shape {tuple(base.shape)}, the call needs {(B, H, Nq, Nk)}")
    positions, key_positions = _positions_of(shape, positions, key_positions)
    rows = _starts_array(shape, starts)
    device = _on_device(table.get_device(), _arg(table, "table", _F32, None),
                        *_positions_args(shape, positions, key_positions), _arg(base, "base", _BF16, None, True))
    bias = torch.empty((B, H, Nq, Nk), dtype=_BF16, device=table.device)
    rc = load().tri_relpos_fwd(shape, rows, table.data_ptr(), _ptr(positions), _ptr(key_positions), _ptr(base),
                               bias.data_ptr(), _raw_stream(device))
    _check("tri_relpos_fwd", rc)
    return bias


def relpos_backward(dbias, starts, two_sided=True, positions=None, key_positions=None, workspace=None,
                    stream=None) -> torch.Tensor:
    """The table's gradient (FP32 [rows, H]) for the gradient dbias [B, H, Nq, Nk] (BF16) of relpos_forward's result."""
    if (other := _other_stream(stream)) is not None:
        return _called_on(other, relpos_backward, dbias, starts, two_sided, positions, key_positions, workspace=workspace)
    if not isinstance(dbias, torch.Tensor):
        raise TypeError(f"dbias must be a torch.Tensor, got {type(dbias).__name__}")
    if dbias.dim() != 4:
        raise ValueError(f"dbias must have four axes (batch, head, query, key), got shape {tuple(dbias.shape)}")
    _axes(*dbias.shape)
    shape = RelposShape(*dbias.shape, len(starts), int(bool(two_sided)))
    positions, key_positions = _positions_of(shape, positions, key_positions)
    rows = _starts_array(shape, starts)
    device = _on_device(dbias.get_device(), _arg(dbias, "dbias", _BF16, None),
                        *_positions_args(shape, positions, key_positions), _arg(workspace, "workspace", None, None, True))
    dtable = torch.empty((shape.rows, shape.H), dtype=_F32, device=dbias.device)
    if workspace is None:
        workspace = _workspace(tri_relpos_bwd_workspace_size(shape), dbias)
    rc = load().tri_relpos_bwd(shape, rows, _ptr(positions), _ptr(key_positions), dbias.data_ptr(), dtable.data_ptr(),
                               _ptr(workspace), _nbytes(workspace), _raw_stream(device))
    _check("tri_relpos_bwd", rc)
    return dtable
