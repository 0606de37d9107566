"""Dense layer and layer norm, forward and backward: binding of libdense.so.

    y = linear(x, w, bias, activation=..., residual=..., preact=z)      bf16, fp16, or int8 with scales
    dx, dw, db = linear_backward(dy, x, w, preact=z, activation=...)
    y, mean, rstd = layer_norm(x, weight, bias)                         bf16, fp16, fp32
    q, scale = layer_norm_i8(x, weight, bias)                           int8 rows for an int8 linear
    dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd)

Argument marshalling only, as in the package's convolution entries: tensors
become the C structures of include/dense.h, and every step runs in the
library's HIP kernels on the current stream (or `stream`).  PyTorch provides
the memory of outputs and workspaces, allocated on the stream the kernels run
on.  Argument errors raise ConvI8Error (a status of conv_i8.h) before any
device work.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

import torch

from . import ConvI8Error, _on_one_gpu, build as _build, status_string

__all__ = ["linear", "linear_plan", "linear_backward", "linear_backward_plan", "layer_norm", "layer_norm_i8",
           "layer_norm_backward", "ACTIVATIONS", "DENSE_LIB_PATH"]

# CONV_I8_DENSE_LIB names another build of the library (the host-sanitizer
# test loads a host-only build with AddressSanitizer through it)
DENSE_LIB_PATH = os.environ.get("CONV_I8_DENSE_LIB") or _build.DENSE_LIB

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

if not os.path.exists(DENSE_LIB_PATH):
    raise ImportError(
        f"{DENSE_LIB_PATH} is not built; run int8_convolution_forward_amd/build.py "
        "(or __graft_entry__.build()) first. There is no fallback implementation.")

lib = ctypes.CDLL(DENSE_LIB_PATH)
# The argument structures hold 8-byte members only, so they are packed with
# struct.pack and passed as bytes: several times cheaper per call than
# ctypes.Structure, which matters for single tokens.
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

_UNKNOWN = 99  # a type code the library refuses
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


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """The tensor as a matrix: its leading dims must merge into one without a copy."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ConvI8Error(3, f"{name}: expected at least one dim")
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.shape[:-1].numel(), t.shape[-1])
    except RuntimeError:
        raise ConvI8Error(8, f"{name}: its leading dims do not merge into rows of one stride") from None


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dim() != 2:
        raise ConvI8Error(3, f"{name}: expected a matrix")
    return t


def _same_gpu(need: int, names: tuple, tensors: tuple) -> int:
    """Index of the one GPU that holds every tensor; past the first `need`,
    None stands for an absent one."""
    try:
        dev = tensors[0].get_device()
        if dev >= 0:
            for i, t in enumerate(tensors):
                if (t is not None or i < need) and t.get_device() != dev:
                    break
            else:
                return dev
    except AttributeError:
        pass
    for name, t in zip(names[:need], tensors):
        if t is None:
            raise TypeError(f"{name}: expected a torch.Tensor, got None")
    _on_one_gpu(**dict(zip(names, tensors)))  # raises, naming the operand
    raise ValueError(f"{names[0]}: expected GPU tensors")


def _activation(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation: {name!r} is none of {', '.join(ACTIVATIONS)}") from None


class _Run:
    """Device and stream of one call: outputs and workspaces are allocated on
    the stream that the kernels run on."""

    def __init__(self, dev: int, stream):
        self.stream = stream
        self.handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
        self.other = dev if dev != torch.cuda.current_device() else None

    def __enter__(self):
        if self.other is not None:
            self.guard = torch.cuda.device(self.other)
            self.guard.__enter__()
        if self.stream is not None:
            self.on = torch.cuda.stream(self.stream)
            self.on.__enter__()
        return self

    def __exit__(self, *exc):
        if self.stream is not None:
            self.on.__exit__(*exc)
        if self.other is not None:
            self.guard.__exit__(*exc)


def _call(entry, size, args: bytes, device, handle) -> None:
    """entry(args, workspace, bytes, stream) with the workspace it asks for."""
    n = _Z()
    _check(size(args, n))
    if n.value:
        ws = torch.empty(n.value, dtype=torch.uint8, device=device)
        _check(entry(args, ws.data_ptr(), n.value, handle))
    else:
        _check(entry(args, None, 0, handle))


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
    written with the value before the activation, which linear_backward takes.
    out, if given, is written and returned; it may be the residual itself.
    """
    dev = _same_gpu(2, ("x", "w", "bias", "residual", "x_scale", "w_scale", "preact", "out"),
                    (x, w, bias, residual, x_scale, w_scale, preact, out))
    act = _activation(activation)
    x2 = x if x.dim() == 2 else _rows(x, "x")
    _matrix(w, "w")
    if x_scale is not None and x_scale.dim() != 1:
        x_scale = _rows(x_scale.unsqueeze(-1), "x_scale").squeeze(-1)
    if residual is not None and residual.dim() != 2:
        residual = _rows(residual, "residual")
    if preact is not None and preact.dim() != 2:
        preact = _rows(preact, "preact")
    with _Run(dev, stream) as run:
        if out is None:
            if out_dtype is None:
                out_dtype = torch.bfloat16 if x.dtype is torch.int8 else x.dtype
            o2 = torch.empty((x2.shape[0], w.shape[0]), dtype=out_dtype, device=x.device)
            y = o2 if x2 is x else o2.view(*x.shape[:-1], w.shape[0])
        else:
            if out_dtype is not None and out.dtype != out_dtype:
                raise ConvI8Error(2, "out: its type is not out_dtype")
            y, o2 = out, _rows(out, "out")
        args = _linear_args(x2, w, bias, act, residual, x_scale, w_scale, preact, o2)
        _call(lib.dense_linear, lib.dense_linear_workspace_size, args, x.device, run.handle)
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
                    stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dw, dbias) of linear for bf16 or fp16 operands of one type.

    g = dy * act'(preact); dx = g w, dw = g^T x, dbias = sum over rows of g.
    preact is what linear kept (not needed without an activation).  The
    gradient of linear's residual is dy.  None stands for what is not needed.
    """
    dev = _same_gpu(3, ("dy", "x", "w", "preact"), (dy, x, w, preact))
    act = _activation(activation)
    dy2, x2 = _rows(dy, "dy"), _rows(x, "x")
    _matrix(w, "w")
    z2 = None if preact is None or act == 0 else _rows(preact, "preact")
    with _Run(dev, stream) as run:
        new = lambda *shape: torch.empty(shape, dtype=dy.dtype, device=dy.device)  # noqa: E731
        dx = new(x2.shape[0], x2.shape[1]) if need_dx else None
        dw = new(w.shape[0], w.shape[1]) if need_dw else None
        db = new(w.shape[0]) if need_dbias else None
        args = _backward_args(dy2, x2, w, z2, act, dx, dw, db)
        _call(lib.dense_linear_backward, lib.dense_linear_backward_workspace_size, args, dy.device, run.handle)
    return (dx if dx is None or x2 is x else dx.view(x.shape)), dw, db


def linear_backward_plan(dy, x, w, preact=None, activation="none", need_dx=True, need_dw=True,
                         need_dbias=True) -> str:
    """How linear_backward would run.  Host-only, matrices only."""
    new = lambda on, *shape: torch.empty(shape, dtype=dy.dtype, device=dy.device) if on else None  # noqa: E731
    args = _backward_args(dy, x, w, preact, _activation(activation), new(need_dx, *x.shape), new(need_dw, *w.shape),
                          new(need_dbias, w.shape[0]))
    buf = ctypes.create_string_buffer(512)
    _check(lib.dense_linear_backward_plan(args, buf, 512))
    return buf.value.decode()


def _norm(x, weight, bias, eps, stream, q8):
    dev = _same_gpu(1, ("x", "weight", "bias"), (x, weight, bias))
    x2 = x if x.dim() == 2 else _rows(x, "x")
    m = x2.shape[0]
    lead = x.shape[:-1]
    with _Run(dev, stream) as run:
        if q8:
            y2 = torch.empty(x2.shape, dtype=torch.int8, device=x.device)
            scale = torch.empty(lead, dtype=torch.float32, device=x.device)
            stats = (*_NO_VEC, *_NO_VEC, scale.data_ptr(), m, 5)
            rest = (scale,)
        else:
            y2 = torch.empty(x2.shape, dtype=x.dtype, device=x.device)
            mean = torch.empty(lead, dtype=torch.float32, device=x.device)
            rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
            stats = (mean.data_ptr(), m, 5, rstd.data_ptr(), m, 5, *_NO_VEC)
            rest = (mean, rstd)
        args = _pack_norm(*_mat(x2), *_mat(y2), *_vec(weight, "weight"), *_vec(bias, "bias"), *stats, eps)
        _check(lib.dense_layer_norm(args, run.handle))
    return (y2 if x2 is x else y2.view(x.shape), *rest)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): layer norm over x's last dim, and the statistics that
    layer_norm_backward takes (fp32, x's leading shape).  x: bf16, fp16 or
    fp32, its last dim contiguous; weight and bias of its type, or None."""
    return _norm(x, weight, bias, eps, stream, False)


def layer_norm_i8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): layer norm's rows as int8, y ~ q * scale[row] with scale =
    max |y| / 127 (fp32, x's leading shape): linear's int8 x and x_scale.  A
    row of zeros has scale 0; a row with a value that is not finite has scale
    NaN and values of no meaning."""
    return _norm(x, weight, bias, eps, stream, True)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, need_params: bool = True, stream=None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dx, dweight, dbias) of layer_norm; the last two are None without
    need_params.  dy has x's shape and type."""
    dev = _same_gpu(2, ("dy", "x", "weight", "mean", "rstd"), (dy, x, weight, mean, rstd))
    dy2, x2 = _rows(dy, "dy"), _rows(x, "x")
    if mean.dim() != 1:
        mean = _rows(mean.unsqueeze(-1), "mean").squeeze(-1)
    if rstd.dim() != 1:
        rstd = _rows(rstd.unsqueeze(-1), "rstd").squeeze(-1)
    with _Run(dev, stream) as run:
        dx2 = torch.empty(x2.shape, dtype=x.dtype, device=x.device)
        dw = db = None
        if need_params:
            dw = torch.empty(x2.shape[1], dtype=x.dtype, device=x.device)
            db = torch.empty(x2.shape[1], dtype=x.dtype, device=x.device)
        args = _pack_norm_backward(*_mat(dy2), *_mat(x2), *_mat(dx2), *_vec(weight, "weight"), *_vec(mean, "mean"),
                                   *_vec(rstd, "rstd"), *_vec(dw, "dweight"), *_vec(db, "dbias"))
        _call(lib.dense_layer_norm_backward, lib.dense_layer_norm_backward_workspace_size, args, x.device, run.handle)
    return (dx2 if x2 is x else dx2.view(x.shape)), dw, db
