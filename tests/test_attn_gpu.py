"""Attention to states of another length, forward and backward, on the GPU against the definition
in 64 bits (attention_reference.py has the bounds and how they come about): head sizes and
types, shared key heads, one token and many, ragged lengths and masks, empty rows, NaN in invisible
places, strides, splits of the keys, streams, graphs and autograd."""
import itertools
import math

import pytest
import torch

import view_deformable_feature_amd as vdf
from attention_reference import BF16, F16, F32, HALF, U, Attention, check
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])

# B, Nq, Nk, H, Hk, D
SHAPES = {
    "one_of_each": (1, 1, 1, 1, 1, 8),
    "one_key": (2, 5, 1, 2, 1, 16),
    "one_query": (2, 1, 70, 4, 4, 32),
    "shared_heads": (2, 3, 129, 8, 2, 64),
    "three_to_a_head": (1, 43, 65, 9, 3, 40),
    "rows_32": (1, 32, 300, 2, 2, 24),
    "rows_33": (1, 33, 300, 2, 2, 24),
    "tile_edges": (1, 128, 128, 1, 1, 128),
    "past_tile_edges": (1, 129, 257, 1, 1, 128),
    "odd": (3, 77, 205, 3, 1, 72),
    "head_96": (1, 61, 99, 2, 1, 96),
    "head_112": (2, 40, 131, 2, 2, 112),
    "head_80": (1, 130, 64, 4, 2, 80),
    "many_keys": (1, 7, 5001, 2, 1, 48),          # split over workgroups
    "wide_32": (4, 130, 150, 64, 64, 32),         # the wide form in each head size
    "wide_64": (3, 200, 67, 48, 48, 64),
    "wide_96": (2, 129, 130, 64, 64, 88),
    "wide_128": (2, 140, 190, 64, 64, 128),
    "wide_shared": (2, 70, 100, 256, 64, 56),
    "wide_split_64": (2, 200, 1000, 20, 20, 64),  # ... with its keys split over workgroups
    "wide_split_96": (1, 220, 1700, 40, 40, 88),
    "wide_split_128": (5, 230, 1500, 9, 9, 128),
    "units_of_eight": (8, 100, 96, 8, 8, 32),
    "units_of_seven": (7, 50, 96, 1, 1, 64),
}


def _inputs(shape, dtype, seed, lens=False, mask=False):
    B, Nq, Nk, H, Hk, D = shape
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, Nq, H, D), generator=gen) * 1.3).to(dtype).cuda()
    k = (torch.randn((B, Nk, Hk, D), generator=gen) + 0.3).to(dtype).cuda()
    v = (torch.randn((B, Nk, Hk, D), generator=gen) + torch.randn(D, generator=gen)).to(dtype).cuda()
    go = torch.randn((B, Nq, H, D), generator=gen).to(dtype).cuda()
    kv = torch.randint(0, Nk + 1, (B,), generator=gen, dtype=torch.int32).cuda() if lens else None
    m = (torch.rand((B, Nk), generator=gen) < 0.7).cuda() if mask else None
    return q, k, v, go, kv, m


def _check(q, k, v, go, kv=None, m=None, scale=None):
    out, lse = vdf.attn_forward(q, k, v, kv, m, scale)
    torch.cuda.synchronize()
    ref = Attention(q, k, v, kv, m, scale)
    ref.check_forward(out, lse)
    grads = vdf.attn_backward(q, k, v, out, lse, go, kv, m, scale)
    torch.cuda.synchronize()
    assert all(g.dtype == q.dtype for g in grads)
    ref.check_backward(grads, go)
    return out, lse, grads


@pytest.mark.parametrize("name", sorted(SHAPES))
@TYPES
def test_shapes(name, dtype):
    say(f"[attn] {name} {SHAPES[name]} {dtype}")
    _check(*_inputs(SHAPES[name], dtype, 10 + sorted(SHAPES).index(name)))


@pytest.mark.parametrize("name", ["one_query", "shared_heads", "odd", "past_tile_edges", "many_keys",
                                  "wide_64", "wide_128", "wide_split_96", "units_of_seven"])
@pytest.mark.parametrize("lens, mask", [(True, False), (False, True), (True, True)],
                         ids=["lens", "mask", "both"])
@TYPES
def test_visible_keys(name, lens, mask, dtype):
    """Ragged lengths, masks, and NaN and infinities in all that is invisible."""
    say(f"[attn] visible {name} {lens} {mask} {dtype}")
    q, k, v, go, kv, m = _inputs(SHAPES[name], dtype, 50 + sorted(SHAPES).index(name), lens, mask)
    B, Nk = k.shape[:2]
    see = torch.ones((B, Nk), dtype=torch.bool, device="cuda")
    if lens:
        see &= torch.arange(Nk, device="cuda") < kv[:, None]
    if mask:
        see &= m
    k[~see] = math.nan
    v[~see] = math.inf
    _check(q, k, v, go, kv, m)


@TYPES
def test_rows_without_a_visible_key(dtype):
    """An entry of length 0, one below 0, one whose mask is all false, beside whole ones; more
    than Nk counts as Nk.  Their out, gradients and their keys' gradients are exactly 0."""
    q, k, v, go, _, _ = _inputs((5, 40, 90, 4, 2, 32), dtype, 90)
    kv = torch.tensor([90, 0, -3, 1000, 90], dtype=torch.int32, device="cuda")
    m = torch.ones((5, 90), dtype=torch.bool, device="cuda")
    m[4] = False
    for t in (k, v):
        t[1:3] = math.nan
        t[4] = math.nan
    out, lse, (dq, dk, dv) = _check(q, k, v, go, kv, m)
    for b in (1, 2, 4):
        assert all((t[b] == 0).all() for t in (out, dq, dk, dv)) and (lse[b] == -math.inf).all()


def test_no_keys_and_no_queries():
    q, k, v, go, _, _ = _inputs((2, 5, 1, 2, 1, 16), BF16, 91)
    k, v = k[:, :0], v[:, :0]
    out, lse = vdf.attn_forward(q, k, v)
    dq, dk, dv = vdf.attn_backward(q, k, v, out, lse, go)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -math.inf).all() and (dq == 0).all() and dk.shape == k.shape
    q, k, v, go, _, _ = _inputs((2, 1, 9, 2, 1, 16), BF16, 92)
    q, go = q[:, :0], go[:, :0]
    out, lse = vdf.attn_forward(q, k, v)
    dq, dk, dv = vdf.attn_backward(q, k, v, out.contiguous(), lse, go.contiguous())
    torch.cuda.synchronize()
    assert out.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    none = vdf.attn_forward(q[:0], k[:0], v[:0])[0]
    assert none.shape == (0, 0, 2, 16)


@TYPES
def test_views_of_one_projection(dtype):
    """q, k and v as views of one projection's output, sequence first, and heads apart; memory
    behind the last token is never read."""
    gen = torch.Generator().manual_seed(93)
    B, N, H, D = 2, 75, 4, 32
    packed = torch.randn((B, N, 3, H, D), generator=gen).to(dtype).cuda()
    q, k, v = packed.unbind(2)
    go = torch.randn((B, N, H, D), generator=gen).to(dtype).cuda()
    _check(q, k, v, go)
    packed = torch.randn((N, B, 3, H, D), generator=gen).to(dtype).cuda()
    q, k, v = (t.transpose(0, 1) for t in packed.unbind(2))
    _check(q, k, v, go)
    packed = torch.randn((B, H, N, 2 * D), generator=gen).to(dtype).cuda()
    packed[..., D:] = math.nan
    _check(q, packed[..., :D].transpose(1, 2), v, go)
    # one entry's states for all
    k1, v1 = (t[:1].expand(B, -1, -1, -1) for t in (k, v))
    _check(q, k1, v1, go)


@TYPES
def test_results_and_gradients_with_strides(dtype):
    """out heads first, into a part of a wider buffer whose rest stays; grad_out heads first."""
    q, k, v, go, _, _ = _inputs((2, 140, 90, 4, 2, 48), dtype, 109)
    buf = torch.full((2, 4, 140, 64), 7.0, dtype=dtype, device="cuda")
    out, lse = vdf.attn_forward(q, k, v, out=buf[..., :48].transpose(1, 2))
    strided = go.transpose(1, 2).contiguous().transpose(1, 2)
    grads = vdf.attn_backward(q, k, v, out, lse, strided)
    torch.cuda.synchronize()
    ref = Attention(q, k, v)
    ref.check_forward(out, lse)
    ref.check_backward(grads, go)
    assert (buf[..., 48:] == 7).all()


@pytest.mark.parametrize("N", [3, 140])
@TYPES
def test_out_in_the_buffer_of_the_projection(dtype, N):
    """out beside q, k and v in one buffer, tokens or heads first: what is there stays."""
    gen = torch.Generator().manual_seed(111)
    B, H, Hk, D = 2, 4, 2, 32
    parts = [H, Hk, Hk, H]
    for heads_first in (False, True):
        shape = (B, sum(parts), N, D) if heads_first else (B, N, sum(parts), D)
        packed = torch.randn(shape, generator=gen).to(dtype).cuda()
        before = packed.clone()
        q, k, v, room = (t.transpose(1, 2) if heads_first else t
                         for t in packed.split(parts, 1 if heads_first else 2))
        want, _ = vdf.attn_forward(q, k, v)
        out, lse = vdf.attn_forward(q, k, v, out=room)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and out.data_ptr() == room.data_ptr()
        Attention(q, k, v).check_forward(out, lse)
        rest = H + 2 * Hk
        assert torch.equal(packed[:, :rest] if heads_first else packed[:, :, :rest],
                           before[:, :rest] if heads_first else before[:, :, :rest])


@TYPES
def test_large_scores(dtype):
    """Scores of hundreds: one key takes all the weight; growing along the keys, so that the
    running maximum moves in every tile."""
    q, k, v, go, _, _ = _inputs((1, 40, 700, 2, 2, 32), dtype, 94)
    grow = torch.linspace(0, 12, 700, device="cuda")[None, :, None, None]
    _check(q, (k + grow).to(dtype), v, go, scale=1.0)
    _check(q, (k - grow).to(dtype), v, go, scale=1.0)


def test_small_and_large_gradients_in_binary16():
    """dP of 1e5 and gradients of 1e-4, whose p (dP - delta) leaves binary16's range at either
    end: results come out as if it did not."""
    q, k, v, go, _, _ = _inputs((1, 70, 500, 2, 1, 64), F16, 95)
    _check(q, k, v, (go * 2.0 ** -13).to(F16))
    q, k, v, go, _, _ = _inputs((1, 70, 900, 2, 1, 64), F16, 96)
    _check(q, (k / 64).to(F16), (v * 100).to(F16), (go * 200).to(F16))


# Queries 256 2^n and, in their second place, 1; keys with as much in the first place and a step of their
# own in the second: scores of 2^n, exact in binary32, that differ by whole steps.
def _far_inputs(shape, dtype, level, seed, step=1.0):
    """(q, k, v, scores [B, H, Nq, Nk] in 64 bits) of scores about 2^level at a scale of 1."""
    B, Nq, Nk, H, Hk, D = shape
    gen = torch.Generator().manual_seed(seed)
    q = torch.zeros((B, Nq, H, D))
    k = torch.zeros((B, Nk, Hk, D))
    q[..., 0] = 2.0 ** (level // 2)
    k[..., 0] = 2.0 ** (level - level // 2)
    q[..., 1] = 1
    k[..., 1] = torch.randint(0, 9, (B, Nk, Hk), generator=gen) * step
    v = torch.randn((B, Nk, Hk, D), generator=gen).to(dtype)
    s = q.double().transpose(1, 2) @ k.double().repeat_interleave(H // Hk, 2).permute(0, 2, 3, 1)
    return q.to(dtype).cuda(), k.to(dtype).cuda(), v.cuda(), s


def _far_levels():
    """Up to where binary16 reaches, 2^15 times 2^15; steps of a unit of the scores' last place in
    binary32, 1 at least."""
    for dtype, most in ((F32, 60), (BF16, 60), (F16, 30)):
        for level in (12, 19, 21, 25, 30, 60):
            if level <= most:
                yield pytest.param(dtype, level, max(1.0, 2.0 ** (level - 23)),
                                   id=f"{str(dtype)[6:]}-{level}")


@pytest.mark.parametrize("dtype, level, step", _far_levels())
@pytest.mark.parametrize("shape", [(2, 3, 90, 4, 2, 32), (1, 2, 9000, 3, 3, 64), (2, 140, 190, 64, 64, 128),
                                   (2, 200, 1000, 20, 20, 64), (1, 1, 1, 1, 1, 8)],
                         ids=["few", "few_split", "wide", "wide_split", "one_key"])
@pytest.mark.parametrize("sign", [1, -1], ids=["up", "down"])
def test_far_scores(dtype, level, step, shape, sign):
    """Scores of 2^12 to 2^60, by whole steps apart: the weights are those of the differences, d.
    Scores are exact here, so what is off is the scale in base 2 (u), the difference's product (u) and
    the exponential (2 u): a weight by (2 d + 3) u of itself, d p at most p (d + 1); in 16 bits by its
    rounding h too, or with 32 rows to a key head by h^2 (binary16: 2^-31 of v); the sums by (n + 32) u."""
    say(f"[attn] far {dtype} 2^{level} {shape} {sign}")
    q, k, v, s = _far_inputs(shape, dtype, level, 301, step)
    q = q * sign
    s = s * sign
    out, lse = vdf.attn_forward(q, k, v, scale=1.0)
    torch.cuda.synchronize()
    B, Nq, Nk, H, Hk, D = shape
    d = s.amax(-1, keepdim=True) - s
    p = torch.exp(-d) / torch.exp(-d).sum(-1, keepdim=True)
    x = v.cpu().double().repeat_interleave(H // Hk, 2).transpose(1, 2)
    want = p @ x
    u, h = 2.0 ** -24, 0.0 if dtype == F32 else 2.0 ** {BF16: -8, F16: -11}[dtype]
    hw = h * h if Nq * (H // Hk) <= 32 else h
    off = p * ((4 * d + 6 + 2 * (Nk + 32)) * u + hw)
    tol = off @ x.abs() + (2.0 ** -31 if dtype == F16 else 0.0) * x.abs().sum(2, keepdim=True)
    check("out", out.transpose(1, 2), want, tol * (1 + h) + h * want.abs() + 2.0 ** -126)
    top = s.amax(-1) + torch.exp(-d).sum(-1).log()
    check("lse", lse, top, top.abs() * 6 * u + (Nk + 32) * u)


@pytest.mark.parametrize("shape", [(2, 3, 900, 4, 2, 32), (1, 2, 9000, 3, 3, 64), (2, 140, 190, 64, 64, 128),
                                   (2, 200, 1000, 20, 20, 64)], ids=["few", "few_split", "wide", "wide_split"])
@pytest.mark.parametrize("sign", [1, -1], ids=["up", "down"])
@TYPES
def test_one_far_score_among_near_ones(dtype, sign, shape):
    """A key in the midst whose score is +-2^25: what its wave, its tile and its split keep meets what
    others do.  It takes all the weight (of the weight, its inverse and the product 3 u), or none, and the
    others share it as if it were invisible."""
    q, k, v, _, _, _ = _inputs(shape, dtype, 306)
    at = shape[2] * 2 // 3
    q[..., 0] = 2.0 ** 13
    k[..., 0] = 0
    k[:, at] = 0
    k[:, at, :, 0] = sign * 2.0 ** 13
    out, lse = vdf.attn_forward(q, k, v, scale=0.5)
    torch.cuda.synchronize()
    if sign > 0:
        x = v[:, at:at + 1].cpu().double().repeat_interleave(shape[3] // shape[4], 2).expand(out.shape)
        check("out", out, x, x.abs() * (3 * U + (0 if dtype == F32 else 2 * HALF[dtype])))
        check("lse", lse, torch.full(lse.shape, 2.0 ** 25, dtype=torch.float64), torch.tensor(4.0).double())
        return
    m = torch.ones(k.shape[:2], dtype=torch.bool, device="cuda")
    m[:, at] = False
    q[..., 0] = 0          # as the other keys see it
    Attention(q, k, v, None, m, 0.5).check_forward(out, lse)


@pytest.mark.parametrize("dtype, level", [(F32, 15), (F32, 20), (F32, 23), (F32, 27), (F32, 34), (F32, 60),
                                          (BF16, 20), (BF16, 34), (BF16, 60), (F16, 20), (F16, 23),
                                          (F16, 26), (F16, 29)])
@pytest.mark.parametrize("Nk", [1, 70])
def test_gradients_of_far_scores(dtype, level, Nk):
    """One key that takes all the weight, scores of +-2^level and up to twice as much.  p comes from
    lse, which is rounded three times on its way to base 2: p is off by a share of at most
    2^(3 u |lse| / log 2) - 1 and 8 u, above 2^22 it is only known to be within 1.  So are the terms of
    grad_v, and with dP and delta the same but for their roundings grad_q and grad_k are next to nothing."""
    say(f"[attn] gradients far {dtype} 2^{level} {Nk}")
    B, Nq, H, D = 2, 90, 3, 16
    gen = torch.Generator().manual_seed(304)
    q, k, v, go, _, _ = _inputs((B, Nq, Nk, H, H, D), dtype, 305)
    q[:], k[:] = 0, 0
    x = (1 + torch.rand((B, Nq, H), generator=gen)) * 2.0 ** (level // 2)
    q[..., 0] = (x * torch.where(torch.rand((B, Nq, H), generator=gen) < 0.5, -1.0, 1.0)).to(dtype).cuda()
    k[..., 0] = 2.0 ** (level - level // 2) / 4          # of invisible keys beside one
    k[:, -1, :, 0] = 2.0 ** (level - level // 2)
    m = torch.zeros((B, Nk), dtype=torch.bool, device="cuda")
    m[:, -1] = True
    out, lse = vdf.attn_forward(q, k, v, None, m, 1.0)
    dq, dk, dv = vdf.attn_backward(q, k, v, out, lse, go, None, m, 1.0)
    torch.cuda.synchronize()
    u, h = 2.0 ** -24, 0.0 if dtype == F32 else 2.0 ** {BF16: -8, F16: -11}[dtype]
    # the key's weight, which need not be a power of two, times v, its inverse, and their product: 3 u
    # (16 bits: the weight's rounding, h, and the result's)
    x = v[:, -1:].cpu().double().expand(out.shape)
    check("out", out, x, x.abs() * (3 * u + 2 * h))
    g = go.cpu().double()
    base2 = lse.cpu().double().abs().transpose(1, 2)[..., None] / math.log(2)
    share = torch.exp2(3 * u * base2) - 1 + 8 * u
    share = torch.where(base2 < 2.0 ** 22, share, 1.0)
    tol = (g.abs() * (share + h + (Nq + 32) * u)).sum(1)
    want = g.sum(1)
    check("grad_v", dv[:, -1], want, tol * (1 + h) + h * want.abs() + 2.0 ** -24)
    assert all(t.isfinite().all() for t in (dq, dk, dv)) and (dk[:, :-1] == 0).all() and (dv[:, :-1] == 0).all()
    # dP - delta: two sums of D products
    less = 2 * (D + 8) * u * (g.abs() * v[:, -1:].cpu().double().abs()).sum(-1, keepdim=True) * 2 * (1 + h)
    check("grad_q", dq, torch.zeros_like(g), less * k[:, -1:].cpu().double().abs() + 2.0 ** -24)


@pytest.mark.parametrize("Nq", [3, 300])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_pass_binary32_once_scaled(Nq, sign):
    """Products of 8 to 90 at a scale of 2^126: the largest alone has weight, lse is infinite."""
    q, k, v, _, _, _ = _inputs((2, Nq, 83, 4, 4, 32), F32, 303)
    q[:], k[:] = 0, 0
    q[..., 0] = sign
    k[..., 0] = torch.arange(8, 91, device="cuda")[:, None]
    out, lse = vdf.attn_forward(q, k, v, scale=2.0 ** 126)
    torch.cuda.synchronize()
    assert torch.equal(out, v[:, 82 if sign > 0 else 0][:, None].expand(out.shape))
    assert (lse == sign * math.inf).all()


@TYPES
def test_far_scores_beside_near_ones(dtype):
    """Rows of scores past 2^20, of ordinary ones and of a growing one in one tile of rows, keys that
    grow along the tiles; and an entry whose keys are all invisible."""
    B, Nq, Nk, D = 2, 150, 700, 32
    for H, rows in ((60, Nq), (2, 5)):
        q, k, v, _, _, _ = _inputs((B, rows, Nk, H, H, D), dtype, 302)
        q[..., 0] = 0
        q[:, ::3, :, 0] = 2.0 ** 14
        q[:, ::3, :, 1:] = 0
        k[..., 0] = (torch.arange(Nk, device="cuda") // 50 * 8 + 2.0 ** 12)[:, None].to(dtype)
        kv = torch.tensor([Nk, 0], dtype=torch.int32, device="cuda")
        out, lse = vdf.attn_forward(q, k, v, kv, scale=0.5)
        torch.cuda.synchronize()
        ref = Attention(q[:, 1::3], k, v, kv, scale=0.5)
        ref.check_forward(out[:, 1::3], lse[..., 1::3])
        # the steps are far apart: the last one's keys share the weight
        first = 650 if dtype != BF16 else int((k[0, :, 0, 0] == k[0, -1, 0, 0]).nonzero()[0])
        n = Nk - first
        mean = v[0, first:].double().mean(0).cpu()
        h = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
        tol = v[0, first:].double().abs().mean(0).cpu() * ((2 * n + 70) * 2.0 ** -24) + h * mean.abs() + 2.0 ** -30
        check("far", out[0, ::3], mean.expand(out[0, ::3].shape), tol)
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("scale", [0.01, 0.5, 3.0])
def test_scale(scale):
    for dtype in (F32, BF16):
        _check(*_inputs((2, 40, 90, 2, 2, 24), dtype, 97), scale=scale)


@pytest.mark.parametrize("scale", [2.0 ** -140, 2.0 ** -120, 2.0 ** 126])
@pytest.mark.parametrize("Nq", [3, 300])
def test_scales_at_the_ends_of_their_range(scale, Nq):
    """Scores that are all equal however large the products, the mean of the values; and scores that
    overflow unless the products are small."""
    q, k, v, _, _, _ = _inputs((2, Nq, 90, 3, 3, 32), F32, 71)
    if scale > 1:
        q, k = q * 2.0 ** -65, k * 2.0 ** -64
    out, lse = vdf.attn_forward(q, k, v, None, None, scale)
    torch.cuda.synchronize()
    Attention(q, k, v, None, None, scale).check_forward(out, lse)


def test_nothing_is_written_past_the_end():
    """Results in buffers with a border, and the workspace's."""
    q, k, v, go, _, _ = _inputs((1, 3, 6000, 2, 1, 40), BF16, 98)
    n = vdf.attn_workspace_size(q, k, v)
    assert n > 0
    ws = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    buf = torch.full((q.numel() + 64,), 7.0, dtype=BF16, device="cuda")
    out, lse = vdf.attn_forward(q, k, v, out=buf[:q.numel()].view(q.shape), workspace=ws[:n])
    torch.cuda.synchronize()
    assert (buf[q.numel():] == 7).all() and (ws[n:] == 0x5a).all()
    Attention(q, k, v).check_forward(out, lse)
    n = vdf.attn_backward_workspace_size(q, k, v)
    ws = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    vdf.attn_backward(q, k, v, out, lse, go, workspace=ws[:n])
    torch.cuda.synchronize()
    assert (ws[n:] == 0x5a).all()


@pytest.mark.parametrize("shape", [(2, 30, 90, 4, 2, 32), (1, 40, 6000, 2, 2, 64), (1, 5000, 40, 2, 1, 24)],
                         ids=["small", "queries_split", "keys_split"])
def test_parts_of_the_gradients(shape):
    q, k, v, go, kv, m = _inputs(shape, BF16, 99, True, True)
    out, lse = vdf.attn_forward(q, k, v, kv, m)
    dq, dk, dv = vdf.attn_backward(q, k, v, out, lse, go, kv, m)
    a = vdf.attn_backward(q, k, v, out, lse, go, kv, m, need_kv=False)
    b = vdf.attn_backward(q, k, v, out, lse, go, kv, m, need_q=False)
    torch.cuda.synchronize()
    assert torch.equal(a[0], dq) and a[1] is None and a[2] is None
    assert b[0] is None and torch.equal(b[1], dk) and torch.equal(b[2], dv)


def test_runs_are_the_same_bit_for_bit():
    for shape in ((2, 1, 9000, 8, 2, 128), (2, 300, 400, 16, 4, 64)):
        q, k, v, go, _, _ = _inputs(shape, BF16, 100)
        out, lse = vdf.attn_forward(q, k, v)
        grads = vdf.attn_backward(q, k, v, out, lse, go)
        for _ in range(3):
            again = vdf.attn_forward(q, k, v)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)
            for g, w in zip(vdf.attn_backward(q, k, v, out, lse, go), grads):
                assert torch.equal(g, w)


@pytest.mark.parametrize("shape", [(2, 1, 9000, 8, 2, 64), (2, 130, 200, 64, 64, 32)],
                         ids=["token", "wide"])
def test_graph_replays_match_eager(shape):
    """Forward and backward captured and replayed, with lengths that change between the replays,
    eager work on the same buffers in between."""
    q, k, v, go, kv, m = _inputs(shape, F16, 101, True, True)
    ws = torch.empty(max(1, vdf.attn_workspace_size(q, k, v)), dtype=torch.uint8, device="cuda")
    bws = torch.empty(vdf.attn_backward_workspace_size(q, k, v), dtype=torch.uint8, device="cuda")

    def step():
        out, lse = vdf.attn_forward(q, k, v, kv, m, workspace=ws)
        return (out, lse, *vdf.attn_backward(q, k, v, out, lse, go, kv, m, workspace=bws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(4):
        kv.copy_(torch.tensor([shape[2] // (n + 1), 17 * n], dtype=torch.int32))
        q.mul_(1.1)
        ws.fill_(0xff)
        bws.fill_(0xff)
        for t in got:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {n}"


def test_two_streams_at_once():
    a = _inputs((2, 200, 700, 8, 4, 64), BF16, 102)
    b = _inputs((1, 1, 9000, 8, 2, 128), BF16, 103)
    want = [vdf.attn_forward(*x[:3]) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(vdf.attn_forward(*x[:3]))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("dtype, shape", list(itertools.product(
    [F32, BF16], [(2, 21, 40, 4, 2, 16), (1, 130, 70, 2, 2, 64)])))
def test_autograd(dtype, shape):
    q, k, v, go, kv, m = _inputs(shape, dtype, 104, True, True)
    kv = kv.clamp_min(5)
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
    out = vdf.cross_attention(*leaves, kv, m)
    (out.float() * go.float()).sum().backward()
    torch.cuda.synchronize()
    Attention(q, k, v, kv, m).check_backward([t.grad for t in leaves], go)
    assert all(t.grad.dtype == dtype for t in leaves)


def test_autograd_of_views_and_shared_states():
    """Queries off alignment and heads first, states shared by the batch entries, whose gradients
    add up; a gradient wanted of the keys alone; a second derivative is refused."""
    gen = torch.Generator().manual_seed(105)
    base = torch.randn((2, 3, 10, 17), generator=gen).cuda().requires_grad_(True)
    k = torch.randn((1, 30, 3, 16), generator=gen).cuda().requires_grad_(True)
    v = torch.randn((1, 30, 3, 16), generator=gen).cuda()
    q = base[..., 1:].transpose(1, 2)
    out = vdf.cross_attention(q, k.expand(2, -1, -1, -1), v.expand(2, -1, -1, -1))
    out.sum().backward()
    torch.cuda.synchronize()
    ref = Attention(q.detach(), k.detach().expand(2, -1, -1, -1), v.expand(2, -1, -1, -1))
    (dq, tq), (dk, tk), _ = ref.backward(torch.ones_like(q))
    check("q.grad", base.grad[..., 1:].transpose(1, 2), dq, tq)
    check("k.grad", k.grad, dk.sum(0, keepdim=True), tk.sum(0, keepdim=True) + 2.0 ** -23 * dk.abs().sum(0, keepdim=True))
    assert (base.grad[..., 0] == 0).all()
    k2 = k.detach().requires_grad_(True)
    g, = torch.autograd.grad(vdf.cross_attention(q.detach(), k2.expand(2, -1, -1, -1),
                                                 v.expand(2, -1, -1, -1)).sum(), k2, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_gradient_against_differences():
    """Central differences of the library's own forward in binary32 along the gradient: with a step
    of h = 2^-7 of unit length the third derivative adds h^2 / 6 times at most (|q| + |k|)^3 / 8
    scale^3 and a few lower terms, below 30 times the loss's magnitude here, and rounding
    2^-18 sum |go| / h."""
    q, k, v, go, _, _ = _inputs((1, 12, 20, 2, 1, 8), F32, 106)
    out, lse = vdf.attn_forward(q, k, v)
    grads = vdf.attn_backward(q, k, v, out, lse, go)
    h = 2.0 ** -7
    for i in range(3):
        t = grads[i] / grads[i].norm()

        def loss(sign):
            x = [q, k, v]
            x[i] = x[i] + sign * h * t
            return (vdf.attn_forward(*x)[0].double() * go.double()).sum()

        want = (loss(1) - loss(-1)) / (2 * h)
        got = (grads[i].double() * t.double()).sum()
        total = float((go.abs().double().sum()))
        assert abs(float(got - want)) <= 30 * h * h / 6 * float(go.abs().max()) * 8 + 2.0 ** -18 * total / h


def test_long_cache():
    """One key head's states past 2^32 bytes from the first batch entry's: 2 x 70000 x 128 heads x
    128 numbers in bfloat16, compared at a few heads and with ragged lengths."""
    B, Nk, H, D = 2, 70000, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(107)
    k = torch.empty((B, Nk, H, D), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    for t in (k, v):
        for b in range(B):
            for r in range(0, Nk, 10000):
                t[b, r:r + 10000] = torch.randn(t[b, r:r + 10000].shape, generator=gen, device="cuda", dtype=BF16)
    q = torch.randn((B, 1, H, D), generator=gen, device="cuda", dtype=BF16)
    kv = torch.tensor([Nk, Nk - 12345], dtype=torch.int32, device="cuda")
    out, lse = vdf.attn_forward(q, k, v, kv)
    torch.cuda.synchronize()
    for h in (0, 77, 127):
        ref = Attention(q[:, :, h:h + 1], k[:, :, h:h + 1], v[:, :, h:h + 1], kv)
        ref.check_forward(out[:, :, h:h + 1], lse[:, h:h + 1])


def test_gradients_of_more_rows_than_threads():
    """2^29 and 160 rows of 8 numbers, all but the first and last tokens' queries and gradients 0: their
    gradients, and the keys', which are those of these tokens."""
    Nq, Nk, H, D, n = (1 << 24) + 5, 70, 32, 8, 40
    gen = torch.Generator().manual_seed(110)
    q, go = (torch.zeros((1, Nq, H, D), dtype=BF16, device="cuda") for _ in range(2))
    for t in (q, go):
        t[:, :n] = torch.randn((1, n, H, D), generator=gen).to(BF16).cuda()
        t[:, -n:] = torch.randn((1, n, H, D), generator=gen).to(BF16).cuda()
    k, v = (torch.randn((1, Nk, H, D), generator=gen).to(BF16).cuda() for _ in range(2))
    out, lse = vdf.attn_forward(q, k, v)
    grads = vdf.attn_backward(q, k, v, out, lse, go)
    torch.cuda.synchronize()

    def ends(t, dim=1):
        return torch.cat([t.narrow(dim, 0, n), t.narrow(dim, Nq - n, n)], dim)

    ref = Attention(ends(q), k, v)
    ref.check_forward(ends(out), ends(lse, 2))
    ref.check_backward((ends(grads[0]), *grads[1:]), ends(go))
    assert not grads[0][:, n:-n].any()


def test_one_device_at_a_time():
    q, k, v, _, kv, m = _inputs((2, 3, 9, 2, 1, 16), F32, 108, True, True)
    with pytest.raises(ValueError, match="GPU"):
        vdf.attn_forward(q, k, v, kv.cpu())
    with pytest.raises(TypeError, match="kv_lens"):
        vdf.attn_forward(q, k, v, kv.long())
    with pytest.raises(TypeError, match="key_mask"):
        vdf.attn_forward(q, k, v, kv, m.to(torch.uint8))
    with pytest.raises(ValueError, match="key_mask"):
        vdf.attn_forward(q, k, v, kv, m[:, :5])
    with pytest.raises(ValueError, match="consecutive"):
        vdf.attn_forward(q, k.transpose(1, 3).contiguous().transpose(1, 3), v)
    with pytest.raises(TypeError, match="k has"):
        vdf.attn_forward(q, k.half(), v.half())
    with pytest.raises(vdf._lib.DAError, match="overlaps"):
        vdf.attn_forward(q, k, v, out=q)
    with pytest.raises(ValueError, match="out"):
        vdf.attn_forward(q, k, v, out=q[:1])
    with pytest.raises(vdf._lib.DAError, match="places of out"):
        vdf.attn_forward(q, k, v, out=torch.empty_like(q)[:1].expand(2, -1, -1, -1))
