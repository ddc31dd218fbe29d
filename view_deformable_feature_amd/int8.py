"""PyTorch binding of the 8-bit products in libdeformagg (include/int8.h): linear layers as
a model is served, for example the one that makes a deformable convolution's
``offset_mask`` from its input or the aggregation's weights from an anchor's features.

``i8_quantize_rows`` makes a layer's 8-bit weights [out_channels, in_channels] with a scale
per output channel once; ``i8_linear`` takes float32, bfloat16 or float16 rows [..., K],
quantises each by its largest magnitude and multiplies; ``i8_matmul`` takes rows that are
codes already; ``i8_norm_linear`` puts a group norm with its activation in front.  These
have no gradients.

Only metadata checks and pointer passing happen here; every step runs in the HIP
kernels of libdeformagg.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib
from .api import _DTYPES, _FLOATS, _need, _ptr, _stream
from .norm import _activation, _gn_problem, _params, _size, _workspace, _ws_args

__all__ = ["i8_quantize_rows", "i8_matmul", "i8_linear", "i8_norm_linear",
           "i8_matmul_workspace_size", "i8_linear_workspace_size",
           "i8_norm_linear_workspace_size"]


def _layer(w, w_scale, bias, dev, K) -> int:
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [out_channels, in_channels] tensor of codes")
    N = w.shape[0]
    _need(w, "w", torch.int8, dev, (N, K))
    _need(w_scale, "w_scale", torch.float32, dev, (N,))
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (N,))
    return N


def _rows(x: torch.Tensor, name: str) -> Tuple[int, int]:
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a [..., K] tensor")
    return math.prod(x.shape[:-1]), x.shape[-1]


def _out(out, out_dtype, shape, dev):
    if out is None:
        return torch.empty(shape, device=dev, dtype=out_dtype)
    _need(out, "out", _FLOATS, dev, shape)
    return out


def _problem(M, K, N, activation, x_dtype, out_dtype) -> _lib.I8Problem:
    if out_dtype not in _DTYPES:
        raise TypeError(f"output dtype must be among {_FLOATS}")
    return _lib.I8Problem(M, K, N, _activation(activation), x_dtype, _DTYPES[out_dtype], 0)


def i8_quantize_rows(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [..., K] int8, scale [...] float32) of x [..., K], row by row."""
    lib = _lib.load()
    M, K = _rows(x, "x")
    dev = x.device
    _need(x, "x", _FLOATS, dev)
    codes = torch.empty(x.shape, device=dev, dtype=torch.int8)
    scale = torch.empty(x.shape[:-1], device=dev, dtype=torch.float32)
    with torch.cuda.device(dev):
        st = lib.i8_quantize_rows(M, K, _DTYPES[x.dtype], _ptr(x), _ptr(codes), _ptr(scale),
                                  _stream(dev))
    _lib.check(st, "i8_quantize_rows")
    return codes, scale


def i8_matmul_workspace_size(rows: int, in_channels: int, out_channels: int) -> int:
    """Bytes of ``workspace`` that ``i8_matmul`` uses."""
    prob = _problem(rows, in_channels, out_channels, "none", 0, torch.float32)
    return _size("i8_matmul_workspace_size", ctypes.byref(prob))


def i8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: str = "none",
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act((a @ w.T) * a_scale * w_scale + bias) [..., N] of codes a [..., K] with a scale per
    row, float32 unless ``out`` / ``out_dtype`` says otherwise."""
    lib = _lib.load()
    M, K = _rows(a, "a")
    dev = a.device
    _need(a, "a", torch.int8, dev)
    _need(a_scale, "a_scale", torch.float32, dev, a.shape[:-1])
    N = _layer(w, w_scale, bias, dev, K)
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    prob = _problem(M, K, N, activation, 0, odt)
    out = _out(out, odt, a.shape[:-1] + (N,), dev)
    need = _size("i8_matmul_workspace_size", ctypes.byref(prob))
    workspace = _workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        st = lib.i8_matmul(ctypes.byref(prob), _ptr(a), _ptr(a_scale), _ptr(w), _ptr(w_scale),
                           _ptr(bias), _ptr(out), *_ws_args(workspace), _stream(dev))
    _lib.check(st, "i8_matmul")
    return out


def i8_linear_workspace_size(rows: int, in_channels: int, out_channels: int,
                             dtype: torch.dtype) -> int:
    """Bytes of ``workspace`` that ``i8_linear`` uses for rows of ``dtype``."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be among {_FLOATS}")
    prob = _problem(rows, in_channels, out_channels, "none", _DTYPES[dtype], torch.float32)
    return _size("i8_linear_workspace_size", ctypes.byref(prob))


def i8_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: str = "none",
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x @ (w * w_scale).T + bias) [..., N] with each row of x [..., K] quantised to 8 bits
    on the way, float32 unless ``out`` / ``out_dtype`` says otherwise."""
    lib = _lib.load()
    M, K = _rows(x, "x")
    dev = x.device
    _need(x, "x", _FLOATS, dev)
    N = _layer(w, w_scale, bias, dev, K)
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    prob = _problem(M, K, N, activation, _DTYPES[x.dtype], odt)
    out = _out(out, odt, x.shape[:-1] + (N,), dev)
    need = _size("i8_linear_workspace_size", ctypes.byref(prob))
    workspace = _workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        st = lib.i8_linear(ctypes.byref(prob), _ptr(x), _ptr(w), _ptr(w_scale), _ptr(bias),
                           _ptr(out), *_ws_args(workspace), _stream(dev))
    _lib.check(st, "i8_linear")
    return out


def i8_norm_linear_workspace_size(x: torch.Tensor, groups: int, out_channels: int) -> int:
    """Bytes of ``workspace`` that ``i8_norm_linear`` uses for x."""
    prob = _gn_problem(x, groups, 0.0, "none", torch.float32)
    return _size("i8_norm_linear_workspace_size", ctypes.byref(prob), int(out_channels))


def i8_norm_linear(x: torch.Tensor, groups: int, norm_weight: Optional[torch.Tensor],
                   norm_bias: Optional[torch.Tensor], w: torch.Tensor, w_scale: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   activation: str = "none", out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The projection [N, ..., out_channels] of act(group norm of x [N, ..., C]), each
    normalised row quantised to 8 bits on the way; ``activation`` stands between norm and
    projection.  float32 unless ``out`` / ``out_dtype`` says otherwise."""
    lib = _lib.load()
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    prob = _gn_problem(x, groups, eps, activation, odt)
    dev, C = x.device, x.shape[-1]
    _need(x, "x", _FLOATS, dev)
    _params(norm_weight, norm_bias, dev, C)
    N = _layer(w, w_scale, bias, dev, C)
    out = _out(out, odt, x.shape[:-1] + (N,), dev)
    need = _size("i8_norm_linear_workspace_size", ctypes.byref(prob), N)
    workspace = _workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        st = lib.i8_norm_linear(ctypes.byref(prob), N, _ptr(x), _ptr(norm_weight), _ptr(norm_bias),
                                _ptr(w), _ptr(w_scale), _ptr(bias), _ptr(out),
                                *_ws_args(workspace), _stream(dev))
    _lib.check(st, "i8_norm_linear")
    return out
