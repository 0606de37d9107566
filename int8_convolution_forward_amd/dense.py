"""Dense layer and layer norm, forward and backward: binding of libdense.so.

    y = linear(x, w, bias, activation=..., residual=..., preact=z)      bf16, fp16, or int8 with scales
    dx, dw, db = linear_backward(dy, x, w, preact=z, activation=...)
    y, mean, rstd = layer_norm(x, weight, bias)                         bf16, fp16, fp32
    q, scale = layer_norm_i8(x, weight, bias)                           int8 rows for an int8 linear
    dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd)

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
from typing import Optional, Tuple

import torch

from . import ConvI8Error, _on_one_gpu, build as _build, status_string

__all__ = ["linear", "linear_plan", "linear_backward", "linear_backward_plan", "layer_norm", "layer_norm_i8",
           "layer_norm_backward", "ACTIVATIONS", "DENSE_LIB_PATH"]

# CONV_I8_DENSE_LIB names another build of the library (the sanitizer test
# loads a host-only build with AddressSanitizer through it)
DENSE_LIB_PATH = os.environ.get("CONV_I8_DENSE_LIB") or _build.DENSE_LIB

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
    "dense_layer_norm", "dense_layer_norm_backward", "dense_layer_norm_backward_workspace_size")))

# The C structures as bytes, for the plans
_UNKNOWN = 99  # a type code the library refuses
_WIDE_G = 256  # DENSE_WIDE_G
_RECORDED = -2  # the native side's: an operand takes part in automatic differentiation
_CODES = {torch.int8: 1, torch.bfloat16: 3, torch.float16: 4, torch.float32: 5}
_NO_MAT = (0, 0, 0, 0, 0, 0)
_NO_VEC = (0, 0, 0)
# pointer, rows, cols, row stride, col stride, type; pointer, n, type
_MAT, _VEC = "Q5q", "Q2q"
_pack_linear = struct.Struct("=" + 5 * _MAT + 3 * _VEC + "q").pack
_pack_linear_backward = struct.Struct("=" + 6 * _MAT + _VEC + "q").pack
_pack_norm = struct.Struct("=" + 2 * _MAT + 5 * _VEC + "d").pack
_pack_norm_backward = struct.Struct("=" + 3 * _MAT + 5 * _VEC).pack


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
