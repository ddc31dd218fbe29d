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
import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib, norm
from ._call import call, maybe, need, scratch, size
from .api import _DTYPES, _FLOATS
from .norm import _activation

__all__ = ["i8_quantize_rows", "i8_matmul", "i8_linear", "i8_norm_linear",
           "i8_matmul_workspace_size", "i8_linear_workspace_size",
           "i8_norm_linear_workspace_size"]


def _layer(w, w_scale, bias, dev, K):
    """(out channels, addresses of codes, scales and bias) of a layer."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [out_channels, in_channels] tensor of codes")
    N = w.shape[:1]
    pw = need(w, "w", torch.int8, dev, N + (K,))
    return (N[0], pw, need(w_scale, "w_scale", torch.float32, dev, N),
            maybe(bias, "bias", torch.float32, dev, N))


def _rows(x, name: str, dtypes):
    """(M, K, type) of rows x [..., K]."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a [..., K] tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {x.dtype}, expected one of {tuple(dtypes)}")
    shape = x.shape
    return math.prod(shape[:-1]), shape[-1]


@functools.lru_cache(maxsize=256)
def _plan(func, M, K, N, activation, x_dtype, out_dtype):
    """(problem, workspace bytes) of a problem's sizes and types; the library only reads the
    problem."""
    if out_dtype not in _DTYPES:
        raise TypeError(f"output dtype must be among {_FLOATS}")
    prob = ctypes.byref(_lib.I8Problem(M, K, N, _activation(activation), x_dtype,
                                       _DTYPES[out_dtype], 0))
    return prob, size(func + "_workspace_size", prob)


@functools.lru_cache(maxsize=256)
def _norm_plan(shape, dtype, groups, eps, activation, N, out_dtype):
    if out_dtype not in _DTYPES:
        raise TypeError(f"output dtype must be among {_FLOATS}")
    prob = ctypes.byref(norm._problem(shape, dtype, groups, eps, activation, out_dtype))
    return prob, size("i8_norm_linear_workspace_size", prob, N)


def i8_quantize_rows(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [..., K] int8, scale [...] float32) of x [..., K], row by row."""
    M, K = _rows(x, "x", _FLOATS)
    dev, shape = x.device, x.shape
    px = need(x, "x", x.dtype, dev, shape)
    codes = torch.empty(shape, device=dev, dtype=torch.int8)
    scale = torch.empty(shape[:-1], device=dev, dtype=torch.float32)
    call("i8_quantize_rows", dev, M, K, _DTYPES[x.dtype], px, codes.data_ptr(), scale.data_ptr())
    return codes, scale


def _product(func, dev, lead, plan, rows, layer, out, odt, workspace):
    """out of a planned product; ``rows``: the addresses that stand for the rows."""
    prob, bytes_needed = plan
    N, pw, ps, pb = layer
    shape = lead + (N,)
    if out is None:
        out = torch.empty(shape, device=dev, dtype=odt)
    po = need(out, "out", odt, dev, shape)
    workspace = scratch(workspace, bytes_needed, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call(func, dev, prob, *rows, pw, ps, pb, po, pws, nws)
    return out


def i8_matmul_workspace_size(rows: int, in_channels: int, out_channels: int) -> int:
    """Bytes of ``workspace`` that ``i8_matmul`` uses."""
    return _plan("i8_matmul", rows, in_channels, out_channels, "none", 0, torch.float32)[1]


def i8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: str = "none",
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act((a @ w.T) * a_scale * w_scale + bias) [..., N] of codes a [..., K] with a scale per
    row, float32 unless ``out`` / ``out_dtype`` says otherwise."""
    M, K = _rows(a, "a", (torch.int8,))
    dev, lead = a.device, a.shape[:-1]
    rows = (need(a, "a", torch.int8, dev, a.shape),
            need(a_scale, "a_scale", torch.float32, dev, lead))
    layer = _layer(w, w_scale, bias, dev, K)
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    plan = _plan("i8_matmul", M, K, layer[0], activation, 0, odt)
    return _product("i8_matmul", dev, lead, plan, rows, layer, out, odt, workspace)


def i8_linear_workspace_size(rows: int, in_channels: int, out_channels: int,
                             dtype: torch.dtype) -> int:
    """Bytes of ``workspace`` that ``i8_linear`` uses for rows of ``dtype``."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be among {_FLOATS}")
    return _plan("i8_linear", rows, in_channels, out_channels, "none", _DTYPES[dtype],
                 torch.float32)[1]


def i8_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: str = "none",
              out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x @ (w * w_scale).T + bias) [..., N] with each row of x [..., K] quantised to 8 bits
    on the way, float32 unless ``out`` / ``out_dtype`` says otherwise."""
    M, K = _rows(x, "x", _FLOATS)
    dev = x.device
    rows = (need(x, "x", x.dtype, dev, x.shape),)
    layer = _layer(w, w_scale, bias, dev, K)
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    plan = _plan("i8_linear", M, K, layer[0], activation, _DTYPES[x.dtype], odt)
    return _product("i8_linear", dev, x.shape[:-1], plan, rows, layer, out, odt, workspace)


def i8_norm_linear_workspace_size(x: torch.Tensor, groups: int, out_channels: int) -> int:
    """Bytes of ``workspace`` that ``i8_norm_linear`` uses for x."""
    _rows(x, "x", _FLOATS)
    return _norm_plan(x.shape, x.dtype, int(groups), 0.0, "none", int(out_channels),
                      torch.float32)[1]


def i8_norm_linear(x: torch.Tensor, groups: int, norm_weight: Optional[torch.Tensor],
                   norm_bias: Optional[torch.Tensor], w: torch.Tensor, w_scale: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   activation: str = "none", out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The projection [N, ..., out_channels] of act(group norm of x [N, ..., C]), each
    normalised row quantised to 8 bits on the way; ``activation`` stands between norm and
    projection.  float32 unless ``out`` / ``out_dtype`` says otherwise."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a [N, ..., C] tensor")
    _, C = _rows(x, "x", _FLOATS)
    dev = x.device
    rows = (need(x, "x", x.dtype, dev, x.shape),
            maybe(norm_weight, "norm_weight", torch.float32, dev, (C,)),
            maybe(norm_bias, "norm_bias", torch.float32, dev, (C,)))
    layer = _layer(w, w_scale, bias, dev, C)
    odt = out.dtype if out is not None else (out_dtype or torch.float32)
    plan = _norm_plan(x.shape, x.dtype, int(groups), float(eps), activation, layer[0], odt)
    return _product("i8_norm_linear", dev, x.shape[:-1], plan, (layer[0],) + rows, layer, out,
                    odt, workspace)
