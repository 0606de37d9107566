"""Dense layer, norms and their companions, forward and backward: binding of libdense.so.

    y = linear(x, w, bias, activation=..., residual=..., preact=z)      bf16, fp16, or int8 with scales
    dx, dw, db = linear_backward(dy, x, w, preact=z, activation=...)
    y, mean, rstd = layer_norm(x, weight, bias)                         bf16, fp16, fp32
    q, scale = layer_norm_i8(x, weight, bias)                           int8 rows for an int8 linear
    dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd)

Around a block in 8-bit floating point, with a scale for each block of 128:

    q, scale, qt, scale_t = quantize_fp8(x, transposed=True)            and dequantize_fp8(q, scale)
    y = linear_fp8(q, w, scale, w_scale, bias, activation=...)
    dx, dw, db = linear_fp8_backward(dy, xt, xt_scale, wt, wt_scale)
    r, y, stats = residual_norm(x, h, weight, gate=..., post_weight=...)   layer norm or rms norm
    r, q, scale = residual_norm_fp8(x, h, weight)                       rows and scales for linear_fp8
    dx, dh, dw, db, dgate, dpost = residual_norm_backward(dr, dy, r, h, stats, weight, ...)
    norm = clip_grad_norm(grads, max_norm)

Argument marshalling only, as in the package's convolution entries: tensors
become the C structures of include/dense.h, and every step runs in the
library's HIP kernels on the current stream, or on `stream`, which then has to
wait for what wrote the operands (they may be freed right after the call).  The
marshalling is native (csrc_dense/bind.cpp), because a call on a single token
lasts only a few microseconds.  PyTorch provides the memory of outputs and
workspaces, allocated on the stream the kernels run on.  Argument errors raise
ConvI8Error (a status of conv_i8.h) before any device work.

Operands may have any strides.  The kernels read most layouts in place or copy
them in their own passes; only leading dims that do not merge into rows of one
stride (a transposed batch), a last dim with a stride where rows have to be
contiguous (layer norm's x, dy, residual and the kept preact) and vectors with
a stride are made contiguous by torch before the call.  `out` and `preact` of
linear have a contiguous last dim and leading dims that merge.

Gradients are the calls above; nothing is recorded for automatic
differentiation.  A tensor that expects it (requires_grad while gradients are
enabled, or a forward-mode tangent) is refused with a RuntimeError, so that no
gradient is lost silently: call under torch.no_grad(), or from the forward and
backward of a torch.autograd.Function.  Tensors given as `out` and `preact`
count as modified in place.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
from typing import Optional, Sequence, Tuple

import torch

from . import ConvI8Error, _on_one_gpu, build as _build, status_string

__all__ = ["linear", "linear_plan", "linear_backward", "linear_backward_plan", "layer_norm", "layer_norm_i8",
           "layer_norm_backward", "quantize_fp8", "dequantize_fp8", "linear_fp8", "linear_fp8_plan", "linear_fp8_backward",
           "linear_fp8_backward_plan", "residual_norm", "residual_norm_fp8", "residual_norm_backward", "clip_grad_norm",
           "ACTIVATIONS", "NORMS", "DENSE_LIB_PATH"]

# CONV_I8_DENSE_LIB names another build of the library (the sanitizer test
# loads a host-only build with AddressSanitizer through it)
DENSE_LIB_PATH = os.environ.get("CONV_I8_DENSE_LIB") or _build.DENSE_LIB

NORMS = {"layer": 0, "rms": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

for _path in (DENSE_LIB_PATH, _build.DENSE_BIND):
    if not os.path.exists(_path):
        raise ImportError(
            f"{_path} is not built; run int8_convolution_forward_amd/build.py "
            "(or __graft_entry__.build()) first. There is no fallback implementation.")

lib = ctypes.CDLL(DENSE_LIB_PATH)
_B, _P, _Z = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t
_ENTRIES = {
    "dense_linear": [_B, _P, _Z, _P],
    "dense_linear_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_linear_plan": [_B, _B, _Z],
    "dense_linear_backward": [_B, _P, _Z, _P],
    "dense_linear_backward_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_linear_backward_plan": [_B, _B, _Z],
    "dense_layer_norm": [_B, _P],
    "dense_layer_norm_backward": [_B, _P, _Z, _P],
    "dense_layer_norm_backward_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_quantize": [_B, _P],
    "dense_dequantize": [_B, _P],
    "dense_linear_fp8": [_B, _P, _Z, _P],
    "dense_linear_fp8_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_linear_fp8_plan": [_B, _B, _Z],
    "dense_linear_fp8_backward": [_B, _P, _Z, _P],
    "dense_linear_fp8_backward_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_linear_fp8_backward_plan": [_B, _B, _Z],
    "dense_residual_norm": [_B, _P],
    "dense_residual_norm_backward": [_B, _P, _Z, _P],
    "dense_residual_norm_backward_workspace_size": [_B, ctypes.POINTER(_Z)],
    "dense_clip_grads": [_B, _P, _Z, _P],
    "dense_clip_grads_workspace_size": [_B, ctypes.POINTER(_Z)],
}
for _name, _types in _ENTRIES.items():
    getattr(lib, _name).argtypes = _types
    getattr(lib, _name).restype = ctypes.c_int

# The native marshalling, and the entries it calls
_loader = importlib.machinery.ExtensionFileLoader("_dense", _build.DENSE_BIND)
_native = importlib.util.module_from_spec(importlib.util.spec_from_loader("_dense", _loader))
_loader.exec_module(_native)
_native.bind(*(ctypes.cast(getattr(lib, n), _P).value for n in (
    "dense_linear", "dense_linear_workspace_size", "dense_linear_backward", "dense_linear_backward_workspace_size",
    "dense_layer_norm", "dense_layer_norm_backward", "dense_layer_norm_backward_workspace_size", "dense_quantize",
    "dense_dequantize", "dense_linear_fp8", "dense_linear_fp8_workspace_size", "dense_linear_fp8_backward",
    "dense_linear_fp8_backward_workspace_size", "dense_residual_norm", "dense_residual_norm_backward",
    "dense_residual_norm_backward_workspace_size", "dense_clip_grads", "dense_clip_grads_workspace_size")))

# The C structures as bytes, for the plans
_UNKNOWN = 99  # a type code the library refuses
_WIDE_G = 256  # DENSE_WIDE_G
_RECORDED = -2  # the native side's: an operand takes part in automatic differentiation
_CODES = {torch.int8: 1, torch.bfloat16: 3, torch.float16: 4, torch.float32: 5, torch.float8_e4m3fn: 6,
          torch.float8_e5m2: 7, torch.float8_e8m0fnu: 8}
_NO_MAT = (0, 0, 0, 0, 0, 0)
_NO_VEC = (0, 0, 0)
# pointer, rows, cols, row stride, col stride, type; pointer, n, type
_MAT, _VEC = "Q5q", "Q2q"
_pack_linear = struct.Struct("=" + 5 * _MAT + 3 * _VEC + "q").pack
_pack_linear_backward = struct.Struct("=" + 6 * _MAT + _VEC + "q").pack
_pack_norm = struct.Struct("=" + 2 * _MAT + 5 * _VEC + "d").pack
_pack_norm_backward = struct.Struct("=" + 3 * _MAT + 5 * _VEC).pack
_pack_quantize = struct.Struct("=" + 5 * _MAT).pack
_pack_dequantize = struct.Struct("=" + 3 * _MAT).pack
_pack_linear_fp8 = struct.Struct("=" + 7 * _MAT + _VEC + "q").pack
_pack_linear_fp8_backward = struct.Struct("=" + 8 * _MAT + _VEC + "2q").pack
_pack_residual_norm = struct.Struct("=" + 6 * _MAT + 7 * _VEC + "2dq").pack
_pack_residual_norm_backward = struct.Struct("=" + 8 * _MAT + 9 * _VEC + "dq").pack
_pack_clip = struct.Struct("=2Qqd1Q").pack


def _check(code: int) -> None:
    if code:
        raise ConvI8Error(code, status_string(code))


def _mat(t: Optional[torch.Tensor]) -> tuple:
    if t is None:
        return _NO_MAT
    r, c = t.shape
    rs, cs = t.stride()
    return (t.data_ptr(), r, c, rs, cs, _CODES.get(t.dtype, _UNKNOWN))


def _vec(t: Optional[torch.Tensor], name: str) -> tuple:
    if t is None:
        return _NO_VEC
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ConvI8Error(8, f"{name}: expected a contiguous vector")
    return (t.data_ptr(), t.shape[0], _CODES.get(t.dtype, _UNKNOWN))


def _refuse(code: int, need: int, **tensors) -> None:
    """Raises for a call that the native side ended: a status, operands that are
    not tensors on one GPU (past the first `need`, None is allowed), or ones
    whose gradients would have to be recorded."""
    if code >= 0:
        raise ConvI8Error(code, status_string(code))
    if code == _RECORDED:
        name = next((n for n, t in tensors.items() if t is not None and t.requires_grad), "an operand")
        raise RuntimeError(f"{name}: expects automatic differentiation, which this call does not record; use "
                           "torch.no_grad() and the backward entries")
    for name in list(tensors)[:need]:
        if tensors[name] is None:
            raise TypeError(f"{name}: expected a torch.Tensor, got None")
    _on_one_gpu(**tensors)
    raise ValueError("expected GPU tensors on one device")


def _activation(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation: {name!r} is none of {', '.join(ACTIVATIONS)}") from None


def _call(entry, stream, *args):
    """entry(*args) with `stream` as the current stream: outputs and workspaces
    are allocated on the stream that the kernels run on, and the memory of the
    operands is not reused before that stream has passed the call."""
    if stream is None:
        return entry(*args)
    x = args[0]
    if isinstance(x, torch.Tensor) and x.is_cuda and x.device != stream.device:
        raise ValueError(f"stream: on {stream.device}, but the operands are on {x.device}")
    with torch.cuda.stream(stream):
        r = entry(*args)
    for t in args:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return r


def _linear_args(x, w, bias, activation, residual, x_scale, w_scale, preact, out) -> bytes:
    return _pack_linear(*_mat(x), *_mat(w), *_mat(out), *_mat(residual), *_mat(preact), *_vec(bias, "bias"),
                        *_vec(x_scale, "x_scale"), *_vec(w_scale, "w_scale"), activation)


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "none",
           residual: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
           w_scale: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
           preact: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act((x w^T) * x_scale[m] * w_scale[n] + bias[n]) + residual, in one pass.

    x [..., K], w [N, K] (its transposed storage is read in place for 16-bit
    types): bf16, fp16, or int8 (exact integer sums, K <= 131071).  bias: N
    values of bf16, fp16 or fp32.  x_scale (one value per row) and w_scale
    (N): fp32, int8 operands only.  The result [..., N] has out_dtype: the
    operands' type by default, bf16 for int8; bf16 and fp16 operands may also
    give fp32.  residual and preact have the result's shape and type; preact is
    written with the value before the activation, which linear_backward takes
    if it is of the operands' type.  out, if given, is written and returned; it
    may be the residual itself.
    """
    y = _call(_native.linear, stream, x, w, bias, _activation(activation), residual, x_scale, w_scale, out_dtype, preact,
              out)
    if type(y) is int:
        _refuse(y, 2, x=x, w=w, bias=bias, residual=residual, x_scale=x_scale, w_scale=w_scale, preact=preact, out=out)
    return y


def linear_plan(x, w, out, bias=None, activation="none", residual=None, x_scale=None, w_scale=None,
                preact=None) -> str:
    """How linear would run (kernel, tile, split, operands copied first).
    Host-only: the tensors may live anywhere, matrices only."""
    args = _linear_args(x, w, bias, _activation(activation), residual, x_scale, w_scale, preact, out)
    buf = ctypes.create_string_buffer(512)
    _check(lib.dense_linear_plan(args, buf, 512))
    return buf.value.decode()


def _backward_args(dy, x, w, preact, activation, dx, dw, dbias) -> bytes:
    return _pack_linear_backward(*_mat(dy), *_mat(x), *_mat(w), *_mat(preact), *_mat(dx), *_mat(dw),
                                 *_vec(dbias, "dbias"), activation)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: Optional[torch.Tensor] = None,
                    activation: str = "none", need_dx: bool = True, need_dw: bool = True, need_dbias: bool = True,
                    stream=None, wide_g: bool = False) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of linear for bf16 or fp16 operands of one type.

    g = dy * act'(preact); dx = g w, dw = g^T x, dbias = sum over rows of g.
    preact is what linear kept (not needed without an activation).  The
    gradient of linear's residual is dy.  None stands for what is not needed.

    The products take g rounded to the operands' type; in fp16, a g below 2^-25
    counts as zero there (small gradients are scaled up by the caller, as for
    every fp16 tensor).  wide_g: they take it as two values of that type, 16
    (bf16) or 22 (fp16) bits and no such loss, at twice the products' work.
    """
    r = _call(_native.linear_backward, stream, dy, x, w, preact, _activation(activation) | (_WIDE_G if wide_g else 0),
              bool(need_dx), bool(need_dw), bool(need_dbias))
    if type(r) is int:
        _refuse(r, 3, dy=dy, x=x, w=w, preact=preact)
    return r


def linear_backward_plan(dy, x, w, preact=None, activation="none", need_dx=True, need_dw=True,
                         need_dbias=True, wide_g=False) -> str:
    """How linear_backward would run.  Host-only, matrices only."""
    new = lambda on, *shape: torch.empty(shape, dtype=dy.dtype, device=dy.device) if on else None  # noqa: E731
    args = _backward_args(dy, x, w, preact, _activation(activation) | (_WIDE_G if wide_g else 0),
                          new(need_dx, *x.shape), new(need_dw, *w.shape), new(need_dbias, w.shape[0]))
    buf = ctypes.create_string_buffer(512)
    _check(lib.dense_linear_backward_plan(args, buf, 512))
    return buf.value.decode()


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): layer norm over x's last dim, and the statistics that
    layer_norm_backward takes (fp32, x's leading shape).  x: bf16, fp16 or
    fp32; weight and bias of its type, or None."""
    r = _call(_native.layer_norm, stream, x, weight, bias, eps, False)
    if type(r) is int:
        _refuse(r, 1, x=x, weight=weight, bias=bias)
    return r


def layer_norm_i8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): layer norm's rows as int8, y ~ q * scale[row] with scale =
    max |y| / 127 (fp32, x's leading shape): linear's int8 x and x_scale.  A
    row of zeros has scale 0; a row with a value that is not finite has scale
    NaN and values of no meaning."""
    r = _call(_native.layer_norm, stream, x, weight, bias, eps, True)
    if type(r) is int:
        _refuse(r, 1, x=x, weight=weight, bias=bias)
    return r


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, need_params: bool = True, stream=None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dweight, dbias) of layer_norm; the last two are None without
    need_params.  dy has x's shape and type."""
    r = _call(_native.layer_norm_backward, stream, dy, x, weight, mean, rstd, bool(need_params))
    if type(r) is int:
        _refuse(r, 2, dy=dy, x=x, weight=weight, mean=mean, rstd=rstd)
    return r



def _norm_kind(name: str) -> int:
    try:
        return NORMS[name]
    except KeyError:
        raise ValueError(f"norm: {name!r} is none of {', '.join(NORMS)}") from None


def quantize_fp8(x: torch.Tensor, block: str = "rows", transposed: bool = False,
                 dtype: torch.dtype = torch.float8_e4m3fn, stream=None) -> Tuple[torch.Tensor, ...]:
    """(q, scale), or (q, scale, qt, scale_t): x [..., K] (bf16, fp16 or fp32) in
    8-bit floating point (float8_e4m3fn or float8_e5m2), x ~ q * scale, with a
    scale for each block, and the same of its transpose [K, rows of x].

    block "rows": 128 values of a row, scale [..., ceil(K / 128)] (what
    linear_fp8 takes for x); "tiles": 128 x 128 values, scale [ceil(rows / 128),
    ceil(K / 128)] (for weights: the transposed copy then holds the same
    values).  A scale is a power of two, in float8_e8m0fnu: the least with which
    the block's largest magnitude is in q's range, 2^-127 at least.  Dividing by it is exact, so
    q is x rounded once.  Values that are not finite become NaN and do not count for
    the scale.
    """
    if block not in ("rows", "tiles"):
        raise ValueError(f"block: {block!r} is none of rows, tiles")
    r = _call(_native.quantize, stream, x, block == "tiles", bool(transposed), dtype)
    if type(r) is int:
        _refuse(r, 1, x=x)
    return r


def dequantize_fp8(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """q * scale in bf16, fp16 or fp32, of what quantize_fp8 gave (either kind of
    block): exact where the value is in the type's range, else rounded to its
    smallest steps (bf16's are 2^-133) or to infinity (3.4e38 is 2^128 in 8 bits)."""
    x = _call(_native.dequantize, stream, q, scale, dtype)
    if type(x) is int:
        _refuse(x, 2, q=q, scale=scale)
    return x


def linear_fp8(x: torch.Tensor, w: torch.Tensor, x_scale: torch.Tensor, w_scale: torch.Tensor,
               bias: Optional[torch.Tensor] = None, activation: str = "none", residual: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, preact: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act((x * x_scale) (w * w_scale)^T + bias[n]) + residual, in one pass.

    x [..., K]: float8_e4m3fn or float8_e5m2, x_scale [..., ceil(K / 128)]; w [N,
    K]: float8_e4m3fn, w_scale [N, ceil(K / 128)] or [ceil(N / 128), ceil(K /
    128)]; scales in float8_e8m0fnu, as quantize_fp8 gives them.  The result [...,
    N] is bf16 by default, or fp16 or fp32; bias, residual, preact and out as in
    linear.

    With out_dtype fp32, products and sums are those of 32 bits (of scaled operands
    of 2^-126 and more, which BF16 holds).  So are those of
    a 16-bit result of up to 32 rows (16 where N > 4096) whose x and w can be read
    in place (K and the strides of their rows multiples of 16, 16-byte aligned
    memory).  Any other 16-bit result is the matrix unit's on 8-bit operands: of
    the products of eight consecutive k, what lies more than 13 bits below the
    largest is cut off before they are summed in 32 bits.  That is below the
    rounding to 16 bits unless a sum cancels; the same row may differ by it between
    calls of few and of many rows.
    """
    y = _call(_native.linear_fp8, stream, x, w, x_scale, w_scale, bias, _activation(activation), residual, out_dtype, preact,
              out)
    if type(y) is int:
        _refuse(y, 4, x=x, w=w, x_scale=x_scale, w_scale=w_scale, bias=bias, residual=residual, preact=preact, out=out)
    return y


def linear_fp8_plan(x, w, x_scale, w_scale, out, bias=None, activation="none", residual=None, preact=None) -> str:
    """How linear_fp8 would run.  Host-only, matrices only."""
    args = _pack_linear_fp8(*_mat(x), *_mat(w), *_mat(out), *_mat(residual), *_mat(preact), *_mat(x_scale), *_mat(w_scale),
                            *_vec(bias, "bias"), _activation(activation))
    buf = ctypes.create_string_buffer(512)
    _check(lib.dense_linear_fp8_plan(args, buf, 512))
    return buf.value.decode()


def linear_fp8_backward(dy: torch.Tensor, xt: Optional[torch.Tensor], xt_scale: Optional[torch.Tensor],
                        wt: Optional[torch.Tensor], wt_scale: Optional[torch.Tensor],
                        preact: Optional[torch.Tensor] = None, activation: str = "none", need_dx: bool = True,
                        need_dw: bool = True, need_dbias: bool = True, g_dtype: torch.dtype = torch.float8_e4m3fn,
                        stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of linear_fp8, from its operands transposed.

    g = dy * act'(preact), in dy's type (bf16 or fp16) [..., N]; dx = Q(g) w, dw =
    Q(g^T) x, dbias = sum over rows of g, all in dy's type.  Q quantises rows to
    g_dtype, a scale for 128 values each: g by its rows for dx, and by its columns
    for dw.  xt [K, rows] and wt [K, N] with their scales are the transposed
    copies that quantize_fp8 gives (float8_e4m3fn, either kind of block); xt is
    not needed without dw, wt not without dx.  The gradient of linear_fp8's
    residual is dy.  Both products are the matrix unit's on 8-bit operands: of the
    products of eight consecutive inner elements, what lies more than 13 bits below
    the largest is cut off before they are summed in 32 bits; dbias sums g in 32
    bits.
    """
    r = _call(_native.linear_fp8_backward, stream, dy, xt, xt_scale, wt, wt_scale, preact, _activation(activation),
              bool(need_dx), bool(need_dw), bool(need_dbias), g_dtype)
    if type(r) is int:
        needed = dict(dy=dy)
        if need_dw:
            needed.update(xt=xt, xt_scale=xt_scale)
        if need_dx:
            needed.update(wt=wt, wt_scale=wt_scale)
        _refuse(r, len(needed), **needed, **{k: v for k, v in dict(xt=xt, xt_scale=xt_scale, wt=wt, wt_scale=wt_scale,
                                                                   preact=preact).items() if k not in needed})
    return r


def linear_fp8_backward_plan(dy, xt, xt_scale, wt, wt_scale, preact=None, activation="none", need_dx=True, need_dw=True,
                             need_dbias=True, g_dtype=torch.float8_e4m3fn) -> str:
    """How linear_fp8_backward would run.  Host-only, matrices only."""
    new = lambda on, *shape: torch.empty(shape, dtype=dy.dtype, device=dy.device) if on else None  # noqa: E731
    k = (wt if need_dx else xt).shape[0] if need_dx or need_dw else 0
    m, n = dy.shape
    args = _pack_linear_fp8_backward(*_mat(dy), *_mat(preact), *_mat(xt), *_mat(xt_scale), *_mat(wt), *_mat(wt_scale),
                                     *_mat(new(need_dx, m, k)), *_mat(new(need_dw, n, k)),
                                     *_vec(new(need_dbias, n), "dbias"), _activation(activation),
                                     _CODES.get(g_dtype, _UNKNOWN))
    buf = ctypes.create_string_buffer(512)
    _check(lib.dense_linear_fp8_backward_plan(args, buf, 512))
    return buf.value.decode()


def residual_norm(x: torch.Tensor, h: Optional[torch.Tensor], weight: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None, scale: float = 1.0, norm: str = "layer", eps: float = 1e-5,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(r, y, stats): the residual connection after a block and the norm before the next, in one pass.

        n = norm(h) * post_weight, or h without it       h: the block's output
        r = scale * x + gate * n, or x without h         rounded to x's type
        y = norm(r) * weight + bias

    norm "layer" is layer norm over the last dim, "rms" the same without the
    mean.  x, h: bf16, fp16 or fp32, everything of one type.  gate: [D], or [...,
    D] of G rows in all, where each is that of 1 / G of x's rows, one after the
    other (a gate for each sequence of a batch).  stats, which
    residual_norm_backward takes, holds mean and rstd of r and, with
    post_weight, of h: fp32, [2 or 4, *x's leading shape] (means of "rms" are 0).

    A row whose squares add up to more than fp32 holds (a deviation of 2^64 /
    sqrt(D), 2.9e17 for D = 4096) has NaN for rstd and is NaN where it is normed,
    as one with an infinity or NaN is.
    """
    r = _call(_native.residual_norm, stream, x, h, weight, bias, gate, post_weight, scale, _norm_kind(norm), eps, False)
    if type(r) is int:
        _refuse(r, 1, x=x, h=h, weight=weight, bias=bias, gate=gate, post_weight=post_weight)
    return r


def residual_norm_fp8(x: torch.Tensor, h: Optional[torch.Tensor], weight: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      post_weight: Optional[torch.Tensor] = None, scale: float = 1.0, norm: str = "layer",
                      eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(r, q, scale): residual_norm with y in float8_e4m3fn and a scale for each
    128 of a row, as quantize_fp8 gives of the unrounded y: linear_fp8's x and
    x_scale."""
    r = _call(_native.residual_norm, stream, x, h, weight, bias, gate, post_weight, scale, _norm_kind(norm), eps, True)
    if type(r) is int:
        _refuse(r, 1, x=x, h=h, weight=weight, bias=bias, gate=gate, post_weight=post_weight)
    return r


def residual_norm_backward(dr: Optional[torch.Tensor], dy: torch.Tensor, r: torch.Tensor, h: Optional[torch.Tensor],
                           stats: torch.Tensor, weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                           post_weight: Optional[torch.Tensor] = None, scale: float = 1.0, norm: str = "layer",
                           need_params: bool = True, stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(dx, dh, dweight, dbias, dgate, dpost_weight) of residual_norm, from the
    gradients of r (None: zero) and y, and what the forward pass gave.  None
    stands for dh, dgate and dpost_weight where h, gate and post_weight are absent
    and, without need_params, for the last four; dweight and dbias are given also
    where there was no weight or bias.  dgate has gate's shape, each of its rows
    summed over the rows that shared it."""
    g = _call(_native.residual_norm_backward, stream, dr, dy, r, h, stats, weight, gate, post_weight, scale,
              _norm_kind(norm), bool(need_params))
    if type(g) is int:
        _refuse(g, 3, dy=dy, r=r, stats=stats, dr=dr, h=h, weight=weight, gate=gate, post_weight=post_weight)
    return g


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   stream=None) -> torch.Tensor:
    """The 2-norm of all values of `grads` together (fp32, on their device, summed
    in 64 bits); they are multiplied by min(1, max_norm / norm), in place or into
    `out`.  An infinity or NaN among the values makes the norm infinite or NaN and
    leaves all of them as they are.  Finite values are scaled also where their norm
    is beyond fp32 and reads as infinity.

    grads: bf16, fp16 or fp32 tensors on one GPU, of any number and shapes, each
    without gaps in memory (in any order of its dims); out: as many, of the same
    types, shapes and strides (of dims longer than one).  Memory that is written may belong to one tensor only.
    """
    grads = list(grads)
    out = None if out is None else list(out)
    if not grads:
        raise ValueError("grads: expected at least one tensor")
    tensors = grads + (out or [])

    def entry(_first, *_rest):
        return _native.clip_grad_norm(grads, max_norm, out)

    r = _call(entry, stream, *tensors)
    if type(r) is int:
        names = {f"grads[{i}]": g for i, g in enumerate(grads)}
        names.update({f"out[{i}]": g for i, g in enumerate(out or [])})
        _refuse(r, len(names), **names)
    return r
