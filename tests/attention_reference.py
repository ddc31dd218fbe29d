"""Attention, its gradients, the rotation and the head norm from the definitions
(include/attention.h, include/rotary.h), in 64 bits on the CPU, and the bounds that the library's
results keep.

Bounds.  u = 2^-24 is half a step of binary32, h half a step of the inputs' type (HALF), relative.

* Scores: D products, exact in 16 bits, add up in binary32: (D + 8) u sum |q k| scale; the scale
  in base 2 and the multiply-add that takes the shift off round once each, by u of the score and of
  the largest one.  The exponential is off by 2 u.  So a weight is off by the share
  e = scale (D + 8) u max |q| |k| + 4 u max |s| + 4 u of itself, and a normalised one by 2 e.
* Sums over n keys: at most n + 32 additions, each off by u of the magnitudes.
* Weights in 16 bits are rounded by h of themselves (with two terms by h^2 and as much as a
  binary16 number below its normal range, 2^-25 at a scale of 2^7); results once, by h.
* p in the gradients comes from the given lse, whose own bound is a share of p.  dP is off by
  (D + 8) u sum |dO v|, delta by as much of sum |dO out| and by sum |dO| times out's bound, since
  out is the rounded one; dS = p (dP - delta) by p times both, its share of p's and h for its
  rounding (binary16: 2^-33 of its largest, which lies at 2^8 or more).
* Sums over rows or keys of these: their bounds' sums, and (n + 32) u of the magnitudes.
"""
import math

import torch

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: U, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -24}


def _heads_first(x, H):
    """[B, N, Hk, D] to [B, H, N, D] in 64 bits."""
    return x.detach().cpu().double().repeat_interleave(H // x.shape[2], 2).transpose(1, 2)


class Attention:
    """few: 32 rows or fewer to a key head, whose weights have two terms."""

    def __init__(self, q, k, v, kv_lens=None, key_mask=None, scale=None):
        B, Nq, H, D = q.shape
        Nk, Hk = k.shape[1:3]
        self.dtype, self.Hk = q.dtype, Hk
        self.scale = float(torch.tensor(1 / math.sqrt(D) if scale is None else scale).float())
        see = torch.ones((B, Nk), dtype=torch.bool)
        if kv_lens is not None:
            see &= torch.arange(Nk) < kv_lens.cpu()[:, None]
        if key_mask is not None:
            see &= key_mask.cpu()
        self.see = see[:, None, None, :]
        self.q = _heads_first(q, H)
        # what stands in invisible places reaches nothing
        keep = see[:, None, :, None]
        self.k = torch.where(keep, _heads_first(k, H), 0.0)
        self.v = torch.where(keep, _heads_first(v, H), 0.0)
        s = self.scale * self.q @ self.k.transpose(2, 3)
        s = torch.where(self.see, s, -math.inf)
        self.lse = torch.logsumexp(s, -1)
        self.lse = torch.where(self.see.any(-1), self.lse, -math.inf)
        p = torch.exp(s - torch.where(self.lse == -math.inf, 0.0, self.lse)[..., None])
        self.p = torch.where(self.see, p, 0.0)
        self.out = self.p @ self.v
        size = torch.where(self.see, s.abs(), 0.0)
        size = size.amax(-1, keepdim=True) if Nk else torch.zeros((B, H, Nq, 1), dtype=torch.float64)
        mag = self.scale * self.q.abs() @ self.k.abs().transpose(2, 3)
        mag = mag.amax(-1, keepdim=True) if Nk else torch.zeros_like(size)
        self.e = (D + 8) * U * mag + 4 * U * size + 4 * U           # [B, H, Nq, 1]
        self.h = 0.0 if q.dtype == F32 else HALF[q.dtype]
        few = Nq * (H // Hk) <= 32
        hw = self.h * self.h if few else self.h
        tiny = 2.0 ** -31 if q.dtype == F16 else 0.0
        n = Nk + 32
        mags = self.p @ self.v.abs()
        self.out_raw = mags * (2 * self.e + hw + 2 * n * U) + tiny * self.v.abs().sum(2, keepdim=True)
        self.out_tol = self.out_raw * (1 + self.h) + self.h * self.out.abs() + TINY[q.dtype]
        self.lse_tol = 2 * self.e[..., 0] + n * U + 4 * U * (torch.where(
            self.lse == -math.inf, 0.0, self.lse).abs() + size[..., 0])

    def check_forward(self, out, lse):
        check("out", out.transpose(1, 2), self.out, self.out_tol)
        empty = self.lse == -math.inf
        got = lse.cpu().double()
        assert torch.equal(got == -math.inf, empty), "rows without a visible key"
        check("lse", torch.where(empty, 0.0, got), torch.where(empty, 0.0, self.lse), self.lse_tol)

    def backward(self, grad_out):
        """(dq, dk, dv) [B, N, heads, D] and the bound of each."""
        B, H, Nq, D = self.q.shape
        Nk = self.k.shape[2]
        do = grad_out.detach().cpu().double().transpose(1, 2)
        p, q, k, v = self.p, self.q, self.k, self.v
        dp = do @ v.transpose(2, 3)
        delta = (do * self.out).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        share = self.e + self.lse_tol[..., None] + 4 * U
        off = p * ((D + 8) * U * (do.abs() @ v.abs().transpose(2, 3))
                   + (D + 8) * U * (do * self.out).abs().sum(-1, keepdim=True)
                   + (do.abs() * self.out_tol).sum(-1, keepdim=True) + 2 * U * delta.abs())
        off = off + ds.abs() * (share + 4 * U + self.h)
        pad = torch.zeros_like(ds)
        if self.dtype == F16:
            pad = pad + 2.0 ** -32 * (off + ds.abs()).amax((2, 3), keepdim=True) if Nk else pad
        off = torch.where(self.see, off + pad, 0.0)
        rows = Nq * (H // self.Hk) + 32

        def per_key_head(t):
            return t.view(B, self.Hk, H // self.Hk, Nk, D).sum(2)

        dq, tq = self.scale * ds @ k, self.scale * (off @ k.abs() + (Nk + 32) * U * ds.abs() @ k.abs())
        dk = per_key_head(self.scale * ds.transpose(2, 3) @ q)
        tk = per_key_head(self.scale * (off + rows * U * ds.abs()).transpose(2, 3) @ q.abs())
        dv = per_key_head(p.transpose(2, 3) @ do)
        tiny = 2.0 ** -39 if self.dtype == F16 else 0.0
        tv = per_key_head((p * (share + self.h + rows * U) + tiny * self.see).transpose(2, 3) @ do.abs())
        out = []
        for g, t in ((dq, tq), (dk, tk), (dv, tv)):
            out.append((g.transpose(1, 2), (t * (1 + self.h) + self.h * g.abs()
                                            + TINY[self.dtype]).transpose(1, 2)))
        return out

    def check_backward(self, grads, grad_out):
        for name, got, (want, tol) in zip(("grad_q", "grad_k", "grad_v"), grads, self.backward(grad_out)):
            if got is not None:
                check(name, got, want, tol)


def check(what, got, ref, tol):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} for {tuple(ref.shape)}"
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        worst = ((got - ref).abs() / tol).nan_to_num(nan=math.inf).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bound, the worst "
                             f"{float(worst):.3g} times it; first at {i}: {float(got[i])} for "
                             f"{float(ref[i])} +- {float(tol.expand_as(ref)[i]):.3g}")


# ---- rotation and head norm --------------------------------------------------------------
#
# * A turn's cosine and sine: the angle's place is exact to far below u, the series are cut
#   below 2^-29 and add up in binary32: 3 u.  The magnitude rounds once.
# * y_a = x_a c - x_b s: a product and a multiply-add: (2 + 4) u of |x_a c| + |x_b s|.
# * r: D squares add up, D u / 2 of it at most (the root halves a share), the quotient, eps and
#   the root 4 u; x r w rounds twice: (D / 2 + 6) u of n.
# * Gradients: g = dn w; the average of g xhat over D: (D + 8) u of the average magnitude besides
#   the shares of dn (6 u of its two magnitudes) and of r.  Sums for the weights over n rows:
#   a lane adds up at most n of them, (n + 16) u of the magnitudes.


def turns(freqs, positions, N):
    """cos and sin [B or 1, N, 1, R / 2]."""
    pos = torch.arange(N)[None] if positions is None else positions.cpu()
    pos = pos if pos.dim() == 2 else pos[None]
    t = pos.double()[:, :, None, None] * freqs.cpu()
    return torch.cos(t), torch.sin(t)


def pairs(x, R, layout):
    """The two halves of the pairs [..., R / 2]."""
    if layout == "interleaved":
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def join(a, b, x, R, layout):
    y = x.clone()
    ya, yb = pairs(y, R, layout)
    ya.copy_(a)
    yb.copy_(b)
    return y


def rotate(x, freqs, positions, layout, magnitude=1.0, inverse=False):
    """(x rotated, the sums of magnitudes) in 64 bits."""
    x = x.detach().cpu().double()
    R = 2 * len(freqs)
    m = float(torch.tensor(magnitude).float())
    c, s = turns(freqs, positions, x.shape[1])
    c, s = m * c, m * (-s if inverse else s)
    a, b = pairs(x, R, layout)
    y = join(a * c - b * s, b * c + a * s, x, R, layout)
    mag = join((a * c).abs() + (b * s).abs() + 2 * abs(m) * U * (a.abs() + b.abs()),
               (b * c).abs() + (a * s).abs() + 2 * abs(m) * U * (a.abs() + b.abs()), x.abs(), R, layout)
    return y, mag + join(abs(m) * b.abs(), abs(m) * a.abs(), torch.zeros_like(x), R, layout)


def rounded(tol, ref, dtype):
    h = 0.0 if dtype == F32 else HALF[dtype]
    return tol * (1 + h) + h * ref.abs() + TINY[dtype]


def norm_rotate(x, w, freqs, positions, layout, eps, magnitude=1.0):
    """(result, bound)."""
    d = x.detach().cpu().double()
    D = d.shape[-1]
    r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + float(torch.tensor(eps).float()))
    n = d * r * (1.0 if w is None else w.cpu().double())
    y, mag = rotate(n, freqs, positions, layout, magnitude)
    return y, rounded((D / 2 + 14) * U * mag, y, x.dtype)


def norm_rotate_grad(x, w, grad, freqs, positions, layout, eps, magnitude=1.0):
    """((dx, bound), (dw, bound))."""
    d = x.detach().cpu().double()
    D = d.shape[-1]
    wt = torch.ones(D).double() if w is None else w.cpu().double()
    r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + float(torch.tensor(eps).float()))
    hat = d * r
    dn, mag = rotate(grad, freqs, positions, layout, magnitude, inverse=True)
    g = dn * wt
    mean = (g * hat).mean(-1, keepdim=True)
    dx = r * (g - hat * mean)
    gm = mag * wt.abs()
    tol = (D + 24) * U * r * (gm + hat.abs() * (gm * hat.abs()).mean(-1, keepdim=True))
    rows = d.shape[0] * d.shape[1] * d.shape[2]
    dw = (dn * hat).sum((0, 1, 2))
    tw = (rows + D / 2 + 32) * U * (mag * hat.abs()).sum((0, 1, 2)) + TINY[F32]
    return (dx, rounded(tol, dx, x.dtype)), (dw, tw)
