"""PyTorch binding of the rotation of heads by their positions' angles, and of the head norm
in the same pass, in libdeformagg (include/rotary.h).

Heads are [B, N, H, D], as a projection's output is once its last dimension is seen as heads;
views with other strides go in as they are (a head's numbers have to be consecutive), and
results may be written in place.  ``freqs`` [R / 2] float64 on the GPU are radians to a step of
position, ``rope_frequencies`` makes them; R = 2 len(freqs) numbers of a head are rotated.
``positions`` are [N] or [B, N] of int32, int64 or float32 (None: 0, 1, 2, ...).  Layouts go by
name: "half" pairs numbers i and i + R / 2, "interleaved" 2 i and 2 i + 1.

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
from ._call import call, need, scratch, size
from .api import _DTYPES, _FLOATS
from .attention import _like, _need_heads, _strides

__all__ = ["rope_frequencies", "rope_forward", "rope_norm_forward", "rope_norm_backward",
           "rope_norm_backward_workspace_size", "RotaryFunction", "NormRotaryFunction", "rotary",
           "norm_rotary"]

_LAYOUTS = {"half": _lib.ROPE_LAYOUT_HALF, "interleaved": _lib.ROPE_LAYOUT_INTERLEAVED}
_POSITIONS = {torch.int32: _lib.ROPE_POS_I32, torch.int64: _lib.ROPE_POS_I64,
              torch.float32: _lib.ROPE_POS_F32}


def rope_frequencies(rotated: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: Optional[int] = None, fast: float = 32.0, slow: float = 1.0,
                     device="cuda") -> Tuple[torch.Tensor, float]:
    """(freqs [rotated / 2] float64 on ``device``, magnitude) for the rotations' ``freqs`` and
    ``magnitude``: pair i turns by base^(-2 i / rotated) to a step.  For contexts ``factor`` times
    the trained ones, ``scaling`` is

    * "linear": all frequencies divided by ``factor``;
    * "base": the base times factor^(R / (R - 2)), so that the first frequency stays and the
      last is divided by ``factor``;
    * "blend": pairs that turn at least ``fast`` times within ``trained`` positions stay, those that
      turn at most ``slow`` times are divided by ``factor``, between the two even over the pairs'
      numbers; magnitude 1 + log(factor) / 10.  The published method is YaRN's, with its bounds of
      the two pairs' numbers (whole ones, 0 and ``rotated`` - 1), which trained weights count on.
    """
    if rotated < 0 or rotated % 2:
        raise ValueError(f"rotated must be even and >= 0, got {rotated}")
    if not base > 1 or not factor >= 1:
        raise ValueError("base must be > 1 and factor >= 1")
    i = torch.arange(rotated // 2, dtype=torch.float64)
    magnitude = 1.0
    if scaling == "base" and rotated > 2:
        base = base * factor ** (rotated / (rotated - 2))
    elif scaling not in ("none", "linear", "base", "blend"):
        raise ValueError(f"scaling must be none, linear, base or blend, got {scaling!r}")
    freqs = base ** (-2 * i / max(rotated, 1))
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "blend":
        if not trained or not fast > slow > 0:
            raise ValueError("blend needs trained positions and fast > slow > 0")

        def number(turns):      # of the pair that turns so often, not a whole one
            return rotated * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(number(fast)), 0)
        high = min(math.ceil(number(slow)), rotated - 1)
        stretched = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        if number(slow) <= 0:   # no pair turns more often
            stretched = torch.ones_like(i)
        freqs = freqs * (1 - stretched) + freqs / factor * stretched
        magnitude = 1 + 0.1 * math.log(factor)
    return freqs.to(device), magnitude


def _layout(name: str) -> int:
    code = _LAYOUTS.get(name)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {name!r}")
    return code


@functools.lru_cache(maxsize=256)
def _problem(D, rotated, eps, magnitude, layout, dtype, flags):
    return ctypes.byref(_lib.RopeProblem(D, rotated, eps, magnitude, _layout(layout), _DTYPES[dtype],
                                         flags, 0))


@functools.lru_cache(maxsize=512)
def _tensor(shape, x_stride, y_stride, pos_type, batched, name):
    """A tensor's description for the library, which only reads it."""
    return ctypes.byref(_lib.RopeTensor(
        *shape[:3], _strides(shape, x_stride, name), _strides(shape, y_stride, name + "'s result"),
        shape[1] if batched else 0, pos_type, 0))


@functools.lru_cache(maxsize=256)
def _backward_size(*args):
    return size("rope_norm_backward_workspace_size", *args)


@functools.lru_cache(maxsize=256)
def _norm_plan(q, q_stride, qo_stride, q_place, k, k_stride, ko_stride, k_place, R, eps, magnitude,
               layout, dtype):
    """(problem, q's description, k's) of shapes, strides and (type of positions, batched), in one
    look: a call of a few microseconds is bound by the host."""
    return (_problem(q[3], R, eps, magnitude, layout, dtype, 0),
            _tensor(q, q_stride, qo_stride, *q_place, "q"),
            None if k is None else _tensor(k, k_stride, ko_stride, *k_place, "k"))


def _check_heads(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError(f"{name} must be a [batch, tokens, heads, head_dim] tensor")
    if x.dtype not in _DTYPES:
        raise TypeError(f"dtypes must be among {_FLOATS}")


def _frequencies(freqs, dev):
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a [R / 2] float64 tensor")
    if freqs.dtype is torch.float64 and freqs.device == dev and freqs.is_contiguous():
        return freqs.data_ptr()
    return need(freqs, "freqs", torch.float64, dev, freqs.shape)


def _weight(w, name, dev, D):
    if w is None:
        return None
    if (isinstance(w, torch.Tensor) and w.dtype is torch.float32 and w.device == dev and w.dim() == 1
            and w.shape[0] == D and w.is_contiguous()):
        return w.data_ptr()
    return need(w, name, torch.float32, dev, (D,))


def _place(positions, name, shape, dev):
    """(address, type, whether each batch entry has its own) of positions."""
    if positions is None:
        return None, _lib.ROPE_POS_INDEX, False
    kind = _POSITIONS.get(positions.dtype) if isinstance(positions, torch.Tensor) else None
    if kind is None:
        raise TypeError(f"{name} must be a tensor of {tuple(_POSITIONS)}")
    at = positions.shape
    batched = len(at) == 2
    if len(at) not in (1, 2):
        raise ValueError(f"{name} must be [N] or [B, N]")
    if (at[-1] == shape[1] and (not batched or at[0] == shape[0]) and positions.device == dev
            and positions.is_contiguous()):
        return positions.data_ptr(), kind, batched
    return need(positions, name, positions.dtype, dev, shape[:2] if batched else shape[1:2]), kind, batched


def _result(out, name, x):
    """out, or a new dense tensor; x's shape and type."""
    if out is None:
        return _like(x)
    if not isinstance(out, torch.Tensor) or out.shape != x.shape:
        raise ValueError(f"{name} must have the shape {tuple(x.shape)}")
    _need_heads(out, name, x.dtype, x.device)
    return out


def rope_forward(x: torch.Tensor, freqs: torch.Tensor, positions: Optional[torch.Tensor] = None,
                 layout: str = "half", magnitude: float = 1.0, inverse: bool = False,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [B, N, H, D] rotated, of x's type; ``inverse`` turns by the angles' negatives (the gradient
    of a rotation).  ``out`` may be x itself, and any view with consecutive heads' numbers."""
    _check_heads(x, "x")
    dev, shape = x.device, x.shape
    px = _need_heads(x, "x", x.dtype, dev)
    pf = _frequencies(freqs, dev)
    pp, kind, batched = _place(positions, "positions", shape, dev)
    out = _result(out, "out", x)
    prob = _problem(shape[3], 2 * freqs.shape[0], 0.0, float(magnitude), layout, x.dtype,
                    _lib.ROPE_FLAG_INVERSE if inverse else 0)
    t = _tensor(shape, x.stride(), out.stride(), kind, batched, "x")
    call("rope_forward", dev, prob, t, px, pp, pf, out.data_ptr())
    return out


def _sides(q, k):
    _check_heads(q, "q")
    if k is not None:
        _check_heads(k, "k")
        if k.dtype != q.dtype or k.shape[3] != q.shape[3]:
            raise ValueError("q and k must have one type and head_dim")


def rope_norm_forward(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                      k_weight: Optional[torch.Tensor], freqs: torch.Tensor,
                      q_positions: Optional[torch.Tensor] = None,
                      k_positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      layout: str = "half", magnitude: float = 1.0,
                      q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q's heads, k's heads) divided by their root mean square, weighted [D] and rotated, in one
    launch; k may be None, and of other batch, tokens and heads than q.  ``q_out`` and ``k_out`` may
    be q and k themselves."""
    _sides(q, k)
    dev, dtype, shape = q.device, q.dtype, q.shape
    pf = _frequencies(freqs, dev)
    pq = _need_heads(q, "q", dtype, dev)
    pw = _weight(q_weight, "q_weight", dev, shape[3])
    pp, *place = _place(q_positions, "q_positions", shape, dev)
    place = tuple(place)
    q_out = _result(q_out, "q_out", q)
    if k is None:
        prob, tq, _ = _norm_plan(shape, q.stride(), q_out.stride(), place, None, None, None, None,
                                 2 * freqs.shape[0], float(eps), float(magnitude), layout, dtype)
        call("rope_norm_forward", dev, prob, tq, pq, pp, pw, q_out.data_ptr(), None, None, None, None,
             None, pf)
        return q_out, None
    ks = k.shape
    pk = _need_heads(k, "k", dtype, dev)
    pkw = _weight(k_weight, "k_weight", dev, ks[3])
    if k_positions is q_positions and ks[:2] == shape[:2]:
        pkp, k_place = pp, place
    else:
        pkp, *k_place = _place(k_positions, "k_positions", ks, dev)
        k_place = tuple(k_place)
    k_out = _result(k_out, "k_out", k)
    prob, tq, tk = _norm_plan(shape, q.stride(), q_out.stride(), place, ks, k.stride(), k_out.stride(),
                              k_place, 2 * freqs.shape[0], float(eps), float(magnitude), layout, dtype)
    call("rope_norm_forward", dev, prob, tq, pq, pp, pw, q_out.data_ptr(), tk, pk, pkp, pkw,
         k_out.data_ptr(), pf)
    return q_out, k_out


def rope_norm_backward_workspace_size(q: torch.Tensor, k: Optional[torch.Tensor]) -> int:
    """Bytes of ``workspace`` that ``rope_norm_backward`` uses."""
    _sides(q, k)
    prob = _problem(q.shape[3], 0, 0.0, 1.0, "half", q.dtype, 0)
    tq, tk = (None if x is None else _tensor(x.shape, x.stride(), x.stride(), 0, False, name)
              for name, x in (("q", q), ("k", k)))
    return _backward_size(prob, tq, tk)


_OF_Q = ("q", "q_weight", "q_positions", "grad_q_out")
_OF_K = ("k", "k_weight", "k_positions", "grad_k_out")


def _backward_side(x, g, w, positions, need_weights, names, dev):
    """(tensor's description, gradient, weight's gradient, addresses) of q or k."""
    name, of_weight, of_positions, of_grad = names
    shape, dtype = x.shape, x.dtype
    if not isinstance(g, torch.Tensor) or g.shape != shape:
        raise ValueError(f"{of_grad} must have {name}'s shape")
    px = _need_heads(x, name, dtype, dev)
    pg = _need_heads(g, of_grad, dtype, dev)
    pw = _weight(w, of_weight, dev, shape[3])
    pp, kind, batched = _place(positions, of_positions, shape, dev)
    dx = _like(x)
    dw = None
    if need_weights:
        dw = (torch.empty(shape[3], device=dev, dtype=torch.float32) if w is None
              else torch.empty_like(w))
    t = _tensor(shape, x.stride(), g.stride(), kind, batched, name)
    return t, dx, dw, (px, pp, pw, pg, dx.data_ptr(), dw.data_ptr() if need_weights else None)


def rope_norm_backward(q: torch.Tensor, k: Optional[torch.Tensor], grad_q_out: torch.Tensor,
                       grad_k_out: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                       k_weight: Optional[torch.Tensor], freqs: torch.Tensor,
                       q_positions: Optional[torch.Tensor] = None,
                       k_positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       layout: str = "half", magnitude: float = 1.0,
                       need_weights: bool = True, workspace: Optional[torch.Tensor] = None):
    """(grad_q, grad_k of the inputs' type, dense; grad_q_weight, grad_k_weight [D] float32), from
    what ``rope_norm_forward`` was given and the gradients of its results.  ``need_weights`` false
    leaves out the weights' part (None in its place)."""
    _sides(q, k)
    dev = q.device
    pf = _frequencies(freqs, dev)
    prob = _problem(q.shape[3], 2 * freqs.shape[0], float(eps), float(magnitude), layout, q.dtype, 0)
    tq, dq, dqw, of_q = _backward_side(q, grad_q_out, q_weight, q_positions, need_weights, _OF_Q, dev)
    if k is None:
        tk, dk, dkw, of_k = None, None, None, (None,) * 6
    else:
        tk, dk, dkw, of_k = _backward_side(k, grad_k_out, k_weight, k_positions, need_weights, _OF_K, dev)
    workspace = scratch(workspace, _backward_size(prob, tq, tk) if need_weights else 0, dev)
    pws, nws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    call("rope_norm_backward", dev, prob, tq, *of_q, tk, *of_k, pf, pws, nws)
    return dq, dk, dqw, dkw


def _consecutive(t):
    return t if t.dim() != 4 or t.shape[3] <= 1 or t.stride(3) == 1 else t.contiguous()


class RotaryFunction(torch.autograd.Function):
    """Autograd wrapper of the rotation: its gradient is the inverse rotation."""

    @staticmethod
    def forward(ctx, x, freqs, positions=None, layout="half", magnitude=1.0):
        ctx.save_for_backward(freqs, positions)
        ctx.conf = (layout, magnitude)
        return rope_forward(_consecutive(x), freqs, positions, layout, magnitude)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        freqs, positions = ctx.saved_tensors
        return (rope_forward(_consecutive(grad_out), freqs, positions, *ctx.conf, inverse=True),
                None, None, None, None)


class NormRotaryFunction(torch.autograd.Function):
    """Autograd wrapper of the head norm and rotation: gradients for q, k and the weights, each in
    its own type."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, freqs, q_positions=None, k_positions=None, eps=1e-6,
                layout="half", magnitude=1.0):
        q, k = _consecutive(q), None if k is None else _consecutive(k)
        w = [None if t is None else t.contiguous().float() for t in (q_weight, k_weight)]
        out = rope_norm_forward(q, k, *w, freqs, q_positions, k_positions, eps, layout, magnitude)
        ctx.save_for_backward(q, k, *w, freqs, q_positions, k_positions)
        ctx.conf = (eps, layout, magnitude)
        ctx.weight_dtypes = tuple(None if t is None else t.dtype for t in (q_weight, k_weight))
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_q, grad_k):
        q, k, qw, kw, freqs, q_positions, k_positions = ctx.saved_tensors
        needs = ctx.needs_input_grad
        gq = _consecutive(grad_q.to(q.dtype))
        gk = None if k is None else _consecutive(grad_k.to(k.dtype))
        dq, dk, dqw, dkw = rope_norm_backward(q, k, gq, gk, qw, kw, freqs, q_positions, k_positions,
                                              *ctx.conf, need_weights=needs[2] or needs[3])
        return (dq if needs[0] else None, dk if needs[1] else None,
                dqw.to(ctx.weight_dtypes[0]) if needs[2] else None,
                dkw.to(ctx.weight_dtypes[1]) if needs[3] and dkw is not None else None,
                None, None, None, None, None, None)


def rotary(x, freqs, positions=None, layout="half", magnitude=1.0):
    """x [B, N, H, D] rotated, differentiable in x."""
    return RotaryFunction.apply(x, freqs, positions, layout, magnitude)


def norm_rotary(q, k, q_weight, k_weight, freqs, q_positions=None, k_positions=None, eps=1e-6,
                layout="half", magnitude=1.0):
    """(q, k) after head norm and rotation, differentiable in q, k and the weights."""
    return NormRotaryFunction.apply(q, k, q_weight, k_weight, freqs, q_positions, k_positions, eps,
                                    layout, magnitude)
