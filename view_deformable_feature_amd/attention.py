"""PyTorch binding of the attention to states of another length in libdeformagg
(include/attention.h).

Queries are [B, Nq, H, D], keys and values [B, Nk, Hk, D] with H a multiple of Hk: the layout
that a projection's output has once its last dimension is seen as heads, so views of one
projection for queries, keys and values go in as they are (their heads' numbers have to be
consecutive, their strides multiples of 16 bytes; so for results that are given).  ``kv_lens`` [B]
int32 says how many keys of each batch entry count, ``key_mask`` [B, Nk] bool which of them; a query
that sees no key gets 0 and an lse of -inf.

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

__all__ = ["attn_forward", "attn_backward", "attn_workspace_size", "attn_backward_workspace_size",
           "CrossAttentionFunction", "cross_attention"]


def _dense(shape):
    D, H = shape[3], max(shape[2], 1)
    return D * H * max(shape[1], 1), D * H, D


def _strides(shape, strides, name):
    """The first three strides as the library takes them; those of dimensions of one place or none,
    which say nothing, as if what they hold were dense."""
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError(f"the numbers of a head of {name} must be consecutive")
    three = ctypes.c_int64 * 3
    return three(*(s if n > 1 else d for n, s, d in zip(shape, strides, _dense(shape))))


@functools.lru_cache(maxsize=256)
def _plan(func, q, k, q_stride, k_stride, v_stride, o_stride, g_stride, scale, dtype):
    """(problem, workspace bytes) of shapes, strides (None: dense) and type; the library only reads
    the problem."""
    B, Nq, H, D = q
    _, Nk, Hk, _ = k
    dense = (*_dense(q), 1)
    prob = ctypes.byref(_lib.AttnProblem(
        B, Nq, Nk, H, Hk, D, _strides(q, q_stride, "q"), _strides(k, k_stride, "k"),
        _strides(k, v_stride, "v"), _strides(q, o_stride or dense, "out"),
        _strides(q, g_stride or dense, "grad_out"),
        1 / math.sqrt(D) if scale is None and D > 0 else scale or 0.0, _DTYPES[dtype], 0, 0))
    return prob, size(func + "_workspace_size", prob)


def _planned(func, q, k, v, scale, out=None, grad_out=None):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [batch, tokens, heads, head_dim] tensor")
    if q.dtype not in _DTYPES:
        raise TypeError(f"dtypes must be among {_FLOATS}")
    shape, ks = q.shape, k.shape
    if ks != v.shape or ks[0] != shape[0] or ks[3] != shape[3]:
        raise ValueError(f"q {tuple(shape)}, k {tuple(ks)} and v {tuple(v.shape)} do not fit together")
    for name, t in (("out", out), ("grad_out", grad_out)):
        if t is not None and (not isinstance(t, torch.Tensor) or t.shape != shape):
            raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return _plan(func, shape, ks, q.stride(), k.stride(), v.stride(),
                 None if out is None else out.stride(),
                 None if grad_out is None else grad_out.stride(),
                 None if scale is None else float(scale), q.dtype)


def _need_heads(t, name, dtype, dev):
    """The address of a strided tensor."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU (got {t.device}); there is no CPU path")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t.data_ptr()


def _like(x):
    """A new dense tensor of x's shape and type."""
    if x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, device=x.device, dtype=x.dtype)


def attn_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> int:
    """Bytes of ``workspace`` that ``attn_forward`` uses."""
    return _planned("attn_forward", q, k, v, None)[1]


def attn_backward_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> int:
    """Bytes of ``workspace`` that ``attn_backward`` uses."""
    return _planned("attn_backward", q, k, v, None)[1]


def _inputs(q, k, v, kv_lens, key_mask):
    dev = q.device
    return (_need_heads(q, "q", q.dtype, dev), _need_heads(k, "k", q.dtype, dev),
            _need_heads(v, "v", q.dtype, dev),
            maybe(kv_lens, "kv_lens", torch.int32, dev, q.shape[:1]),
            maybe(key_mask, "key_mask", torch.bool, dev, k.shape[:2]))


def attn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 kv_lens: Optional[torch.Tensor] = None, key_mask: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [B, Nq, H, D] of q's type, lse [B, H, Nq] float32).  ``scale`` is 1 / sqrt(D) unless
    given; ``out`` may be any view whose places do not overlap."""
    prob, bytes_needed = _planned("attn_forward", q, k, v, scale, out)
    dev, shape = q.device, q.shape
    pq, pk, pv, pl, pm = _inputs(q, k, v, kv_lens, key_mask)
    if out is None:
        out = _like(q)
    po = _need_heads(out, "out", q.dtype, dev)
    lse = torch.empty((shape[0], shape[2], shape[1]), device=dev, dtype=torch.float32)
    workspace = scratch(workspace, bytes_needed, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call("attn_forward", dev, prob, pq, pk, pv, pl, pm, po, lse.data_ptr(), pws, nws)
    return out, lse


def attn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                  lse: torch.Tensor, grad_out: torch.Tensor, kv_lens: Optional[torch.Tensor] = None,
                  key_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  need_q: bool = True, need_kv: bool = True,
                  workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_q, grad_k, grad_v) of the inputs' shapes and type, dense, from what ``attn_forward``
    was given and returned; ``need_q`` and ``need_kv`` false leave out that part (None in its
    place)."""
    prob, bytes_needed = _planned("attn_backward", q, k, v, scale, out, grad_out)
    dev, shape, dtype = q.device, q.shape, q.dtype
    pq, pk, pv, pl, pm = _inputs(q, k, v, kv_lens, key_mask)
    po = _need_heads(out, "out", dtype, dev)
    ps = need(lse, "lse", torch.float32, dev, (shape[0], shape[2], shape[1]))
    pg = _need_heads(grad_out, "grad_out", dtype, dev)
    dq = _like(q) if need_q else None
    dk, dv = (_like(k), _like(v)) if need_kv else (None, None)
    pdq = dq.data_ptr() if need_q else None
    pdk, pdv = (dk.data_ptr(), dv.data_ptr()) if need_kv else (None, None)
    workspace = scratch(workspace, bytes_needed, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call("attn_backward", dev, prob, pq, pk, pv, po, ps, pg, pl, pm, pdq, pdk, pdv, pws, nws)
    return dq, dk, dv


def _fits(t):
    """t itself where the kernels take its strides and place, else a dense copy."""
    per = 16 // t.element_size()
    if (t.dim() == 4 and (t.shape[3] > 1 and t.stride(3) != 1 or t.data_ptr() % 16
                          or any(n > 1 and s % per for n, s in zip(t.shape[:3], t.stride())))):
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


class CrossAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: gradients for q, k and v, each in its own type."""

    @staticmethod
    def forward(ctx, q, k, v, kv_lens=None, key_mask=None, scale=None):
        q, k, v = _fits(q), _fits(k), _fits(v)
        out, lse = attn_forward(q, k, v, kv_lens, key_mask, scale)
        ctx.save_for_backward(q, k, v, out, lse, kv_lens, key_mask)
        ctx.scale = scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        q, k, v, out, lse, kv_lens, key_mask = ctx.saved_tensors
        need_q, need_k, need_v = ctx.needs_input_grad[:3]
        dq, dk, dv = attn_backward(q, k, v, out, lse, _fits(grad_out.to(q.dtype)),
                                   kv_lens, key_mask, ctx.scale, need_q=need_q,
                                   need_kv=need_k or need_v)
        return dq, dk if need_k else None, dv if need_v else None, None, None, None


def cross_attention(q, k, v, kv_lens=None, key_mask=None, scale=None):
    """Attention of q [B, Nq, H, D] to k, v [B, Nk, Hk, D], differentiable in q, k and v."""
    return CrossAttentionFunction.apply(q, k, v, kv_lens, key_mask, scale)
