"""Group norm, its gradients, 8-bit codes and their products from the definitions
(include/group_norm.h, include/int8.h), in 64 bits on the CPU, and the bounds that the
library's 32-bit results keep.

Bounds.  u = 2^-24 is half a step of binary32, relative.  With d = x - mean:

* normalised value z = d * rstd * w + b: mean is rounded once (u |mean|), d once, rstd, its
  product with w and the multiply-add once each, and the statistics' sums run over at
  most ~32 values in a row of a thread and ~10 joins (each value's deviation is taken from
  a value of its own channel, so the error is a share of deviations): 64 u of the
  magnitudes zmag = |d rstd w| + |mean| rstd |w| + |b| + |w| covers them, the |w| standing
  for a mean that is off by a share of the standard deviation.
* activations: slopes are below 1.13, and the hardware's exponential and reciprocal or the
  error function add less than 8 u |z|: doubling the bound on z covers both.
* gradients: act'' is below 0.8, so dz = grad act'(z) is off by 64 u |grad| (1 + zmag); sums
  over rows add 64 u of the sum of magnitudes.  Where |z| is below its bound, the derivative
  of the rectifier is 0 or 1: the whole |grad| is allowed for there.
* products: the integer sum is exact; its conversion, the two scales, the bias and the
  activation round once each: 8 u of the magnitudes.
* a result stored in 16 bits: half a step of it more, eps / 2.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


class Norm:
    """Everything of one normalisation of x [N, S, C], in 64 bits."""

    def __init__(self, x, G, w, b, eps, name):
        self.x = x = x.detach().cpu().double()
        N, S, C = x.shape
        self.name, self.G = name, G
        self.w = torch.ones(C).double() if w is None else w.detach().cpu().double()
        self.b = torch.zeros(C).double() if b is None else b.detach().cpu().double()
        v = x.reshape(N, S, G, C // G)
        m = v.mean((1, 3))
        d = v - m[:, None, :, None]
        var = (d * d).mean((1, 3))
        self.mean, self.rstd = m, 1 / torch.sqrt(var + float(np.float32(eps)))
        self.rs = self._per_channel(self.rstd)
        self.xhat = (d.reshape(N, S, C) * self.rs)
        self.z = self.xhat * self.w + self.b
        mean = self._per_channel(self.mean)
        self.zmag = ((self.xhat * self.w).abs() + mean.abs() * self.rs * self.w.abs() + self.b.abs()
                     + self.w.abs())
        self.ztol = 64 * U * self.zmag
        self.y = act(self.z, name)

    def _per_channel(self, g):
        N, S, C = self.x.shape
        return g[:, None, :].expand(N, 1, self.G).repeat_interleave(C // self.G, 2)

    def out_tol(self, dtype):
        return 2 * self.ztol + HALF[dtype] * self.y.abs() * (0 if dtype == torch.float32 else 1) + TINY[dtype]

    def stat_tols(self):
        std = 1 / self.rstd
        return 64 * U * (self.mean.abs() + std), 64 * U * self.rstd

    def backward(self, dy):
        """(dx, dw, db), and the bound of each before its rounding to 16 bits."""
        N, S, C = self.x.shape
        dy = dy.detach().cpu().double()
        dz = dy * act_grad(self.z, self.name)
        e = 64 * U * dy.abs() * (1 + self.zmag)                    # bound of dz
        if self.name == "relu":
            e = e + torch.where(self.z.abs() <= self.ztol, dy.abs(), torch.zeros_like(dy))

        def group_mean(t):
            return self._per_channel(t.reshape(N, S, self.G, C // self.G).mean((1, 3)))

        wdz, we = dz * self.w, e * self.w.abs()
        m1, m2 = group_mean(wdz), group_mean(wdz * self.xhat)
        dx = self.rs * (wdz - m1 - self.xhat * m2)
        xe = 64 * U * (self.xhat.abs() + self._per_channel(self.mean).abs() * self.rs + 1)   # bound of xhat
        e1 = group_mean(we + 64 * U * wdz.abs())
        e2 = group_mean(we * self.xhat.abs() + wdz.abs() * (xe + 64 * U * self.xhat.abs()))
        tx = self.rs * (we + e1 + self.xhat.abs() * e2 + xe * m2.abs()
                        + 64 * U * (wdz.abs() + m1.abs() + (self.xhat * m2).abs()))
        dw, db = (dz * self.xhat).sum((0, 1)), dz.sum((0, 1))
        tw = (e * self.xhat.abs() + dz.abs() * (xe + 64 * U * self.xhat.abs())).sum((0, 1))
        tb = (e + 64 * U * dz.abs()).sum((0, 1))
        return (dx, dw, db), (tx + 2.0 ** -149, tw + 2.0 ** -149, tb + 2.0 ** -149)


def rounded(tol, ref, dtype):
    """The bound of a 16-bit result whose value before rounding is within tol."""
    return tol if dtype == torch.float32 else tol * (1 + 2 * HALF[dtype]) + HALF[dtype] * ref.abs() + TINY[dtype]


def codes(x):
    """(codes, scale) of the rows of x [M, K], by the definition's binary32 steps."""
    x = x.detach().cpu().float().numpy()
    big = np.abs(x).max(axis=1)
    q = np.zeros(x.shape, np.int8)
    scale = np.zeros(len(x), np.float32)
    for m in range(len(x)):
        if not np.isfinite(big[m]):
            scale[m] = np.nan
        elif big[m] >= np.float32(2.0 ** -100):
            inverse = np.float32(127) / big[m]
            q[m] = np.rint(x[m] * inverse).astype(np.int8)
            scale[m] = big[m] / np.float32(127)
    return torch.from_numpy(q), torch.from_numpy(scale)


def product(a, a_scale, w, w_scale, bias, name):
    """(out, bound before rounding to 16 bits) of codes."""
    s = a.cpu().double() @ w.cpu().double().t()
    y = s * a_scale.cpu().double()[:, None] * w_scale.cpu().double()[None, :]
    mag = y.abs()
    if bias is not None:
        y = y + bias.cpu().double()
        mag = mag + bias.cpu().double().abs()
    return act(y, name), 8 * U * mag + 8 * U * y.abs() + 2.0 ** -140


def check(what, got, ref, tol):
    got = got.detach().cpu().double().reshape(ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        worst = ((got - ref).abs() / tol).nan_to_num(nan=float("inf")).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bound, the worst "
                             f"{float(worst):.3g} times it; first at {i}: {float(got[i])} for "
                             f"{float(ref[i])} +- {float(tol.expand_as(ref)[i]):.3g}")


def gelu_tols(z):
    """Bounds of GELU and of its derivative in binary32 at exactly known z [64 bits].  Phi's own is
    (24 + 2 z^2) u of itself (act_device.h): 1 of the polynomial, 3 of its argument (a multiply-
    add and the hardware's reciprocal) times 2.8, by which f changes with t at the most, 2 for
    each rounding of the sum, which its last terms carry, 2 of the exponential and 3 of the
    products; z^2 for z * z / 2, z^2 for its factor log2(e), twice rounded.  GELU adds the product
    with z, the density half of the exponential's and two products."""
    phi = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    rel = (24 + 2 * z * z) * U
    return ((rel + U) * (z * phi).abs() + 2.0 ** -149,
            rel * phi + (rel + 4 * U) * (z * density).abs() + 2 * U * act_grad(z, "gelu").abs()
            + 2.0 ** -149)
