"""PyTorch binding of the group norm with an activation in libdeformagg
(include/group_norm.h).

Maps are channels last, [N, ..., C] with any number of dimensions between (they are the
rows of an image): the layout ``dcn_forward`` and the aggregation work in, so a
normalisation between two of them copies nothing.  Activations go by name: "none", "relu",
"silu", "gelu" (z times the normal distribution function of z).

Only metadata checks and pointer passing happen here; every step runs in the HIP
kernels of libdeformagg.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._call import call, maybe, need, scratch, size
from .api import _DTYPES, _FLOATS

__all__ = ["gn_forward", "gn_backward", "gn_workspace_size", "gn_backward_workspace_size",
           "GroupNormActFunction", "group_norm_act"]

_ACTIVATIONS = {"none": _lib.DA_ACT_NONE, "relu": _lib.DA_ACT_RELU, "silu": _lib.DA_ACT_SILU,
                "gelu": _lib.DA_ACT_GELU}


def _activation(name: str) -> int:
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {name!r}")
    return code


def _problem(shape, dtype, groups, eps, activation, out_dtype) -> _lib.GNProblem:
    return _lib.GNProblem(shape[0], math.prod(shape[1:-1]), shape[-1], groups, eps,
                          _activation(activation), _DTYPES[dtype], _DTYPES[out_dtype], 0, 0)


@functools.lru_cache(maxsize=256)
def _plan(func, shape, dtype, groups, eps, activation, out_dtype):
    """(problem, workspace bytes) of a problem's sizes and types; the library only reads the
    problem."""
    prob = ctypes.byref(_problem(shape, dtype, groups, eps, activation, out_dtype))
    return prob, size(func + "_workspace_size", prob)


def _planned(func, x, groups, eps, activation, out_dtype):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a [N, ..., C] tensor")
    if x.dtype not in _DTYPES or out_dtype not in _DTYPES:
        raise TypeError(f"input / output dtypes must be among {_FLOATS}")
    return _plan(func, x.shape, x.dtype, int(groups), float(eps), activation, out_dtype)


def gn_workspace_size(x: torch.Tensor, groups: int) -> int:
    """Bytes of ``workspace`` that ``gn_forward`` uses for x."""
    return _planned("gn_forward", x, groups, 0.0, "none", x.dtype)[1]


def gn_backward_workspace_size(x: torch.Tensor, groups: int,
                               grad_dtype: Optional[torch.dtype] = None) -> int:
    """Bytes of ``workspace`` that ``gn_backward`` uses for x and a grad_out of ``grad_dtype``
    (x's type unless given)."""
    return _planned("gn_backward", x, groups, 0.0, "none", grad_dtype or x.dtype)[1]


def gn_forward(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, activation: str = "none",
               out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
               workspace: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(out [N, ..., C], mean [N, G] float32, rstd [N, G] float32): act of the normalised,
    scaled and shifted x.  out has x's type unless ``out`` / ``out_dtype`` says otherwise;
    ``out`` may be x itself."""
    odt = out.dtype if out is not None else (out_dtype or x.dtype)
    prob, bytes_needed = _planned("gn_forward", x, groups, eps, activation, odt)
    dev, shape = x.device, x.shape
    C = shape[-1:]
    px = need(x, "x", x.dtype, dev, shape)
    pw = maybe(weight, "weight", torch.float32, dev, C)
    pb = maybe(bias, "bias", torch.float32, dev, C)
    if out is None:
        out = torch.empty(shape, device=dev, dtype=odt)
    po = need(out, "out", odt, dev, shape)
    mean = torch.empty((shape[0], int(groups)), device=dev, dtype=torch.float32)
    rstd = torch.empty((shape[0], int(groups)), device=dev, dtype=torch.float32)
    workspace = scratch(workspace, bytes_needed, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call("gn_forward", dev, prob, px, pw, pb, po, mean.data_ptr(), rstd.data_ptr(), pws, nws)
    return out, mean, rstd


def gn_backward(x: torch.Tensor, grad_out: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                groups: int, weight: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, activation: str = "none",
                grad_x: Optional[torch.Tensor] = None, need_x: bool = True,
                need_params: bool = True, workspace: Optional[torch.Tensor] = None
                ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_x of x's type, grad_weight [C] float32, grad_bias [C] float32), from what
    ``gn_forward`` was given and returned.  ``grad_x`` may be grad_out itself; ``need_x`` and
    ``need_params`` false leave out that part (None in its place)."""
    if not isinstance(grad_out, torch.Tensor) or grad_out.dtype not in _DTYPES:
        raise TypeError(f"grad_out must be a tensor of one of {_FLOATS}")
    prob, bytes_needed = _planned("gn_backward", x, groups, 0.0, activation, grad_out.dtype)
    dev, shape = x.device, x.shape
    C, stats = shape[-1:], (shape[0], int(groups))
    px = need(x, "x", x.dtype, dev, shape)
    pg = need(grad_out, "grad_out", grad_out.dtype, dev, shape)
    pm = need(mean, "mean", torch.float32, dev, stats)
    pr = need(rstd, "rstd", torch.float32, dev, stats)
    pw = maybe(weight, "weight", torch.float32, dev, C)
    pb = maybe(bias, "bias", torch.float32, dev, C)
    if grad_x is None and need_x:
        grad_x = torch.empty(shape, device=dev, dtype=x.dtype)
    pgx = maybe(grad_x, "grad_x", x.dtype, dev, shape)
    gw = torch.empty(C, device=dev, dtype=torch.float32) if need_params else None
    gb = torch.empty(C, device=dev, dtype=torch.float32) if need_params else None
    pgw, pgb = (gw.data_ptr(), gb.data_ptr()) if need_params else (None, None)
    workspace = scratch(workspace, bytes_needed, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call("gn_backward", dev, prob, px, pg, pm, pr, pw, pb, pgx, pgw, pgb, pws, nws)
    return grad_x, gw, gb


class GroupNormActFunction(torch.autograd.Function):
    """Autograd wrapper: gradients for x, weight and bias, each in its own type (the
    parameters' sums are formed in float32)."""

    @staticmethod
    def forward(ctx, x, groups, weight=None, bias=None, eps=1e-5, activation="none",
                out_dtype=None):
        x = x.contiguous()
        w = None if weight is None else weight.contiguous().float()
        b = None if bias is None else bias.contiguous().float()
        out, mean, rstd = gn_forward(x, groups, w, b, eps, activation, out_dtype=out_dtype)
        ctx.save_for_backward(x, w, b, mean, rstd)
        ctx.conf = (groups, activation)
        ctx.param_dtypes = tuple(None if p is None else p.dtype for p in (weight, bias))
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        x, w, b, mean, rstd = ctx.saved_tensors
        groups, activation = ctx.conf
        if grad_out.dtype not in _DTYPES:
            grad_out = grad_out.float()
        need_x, _, need_w, need_b = ctx.needs_input_grad[:4]
        gx, gw, gb = gn_backward(x, grad_out.contiguous(), mean, rstd, groups, w, b, activation,
                                 need_x=need_x, need_params=need_w or need_b)
        wt, bt = ctx.param_dtypes
        return (gx, None, gw.to(wt) if need_w else None, gb.to(bt) if need_b else None,
                None, None, None)


def group_norm_act(x, groups, weight=None, bias=None, eps=1e-5, activation="none", out_dtype=None):
    """act(group norm of x [N, ..., C]), differentiable in x, weight and bias."""
    return GroupNormActFunction.apply(x, groups, weight, bias, eps, activation, out_dtype)
