"""The rotation of heads, and the head norm with it, forward and backward, on the GPU against the
definition in 64 bits (attention_reference.py has the bounds): layouts, parts of a head, sizes
that fill vectors and sizes that do not, kinds of positions, views, in place, graphs and
autograd."""
import math

import pytest
import torch

import view_deformable_feature_amd as vdf
from attention_reference import (BF16, F16, F32, HALF, U, check, norm_rotate, norm_rotate_grad, rotate,
                                 rounded)
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
LAYOUTS = pytest.mark.parametrize("layout", ["half", "interleaved"])
EPS = 1e-6

# B, N, H, D, R
SHAPES = {
    "one": (1, 1, 1, 2, 2),
    "one_number": (1, 3, 2, 1, 0),
    "head_128": (2, 37, 5, 128, 128),
    "head_64": (3, 20, 3, 64, 64),
    "part": (2, 30, 4, 128, 64),
    "part_80": (2, 33, 9, 80, 40),
    "three_pairs": (2, 17, 2, 24, 6),            # single numbers
    "five_pairs": (1, 40, 3, 40, 10),
    "odd_head": (2, 11, 3, 33, 16),
    "pairs_of_two": (1, 19, 2, 36, 36),
    "none_rotated": (1, 9, 2, 16, 0),
    "widest": (1, 5, 2, 512, 512),
    "widest_pairs": (1, 5, 2, 508, 508),
    "widest_single": (1, 5, 2, 511, 510),
    "one_token_many_heads": (1, 1, 70, 128, 128),
    "many_tokens": (4, 5000, 2, 64, 32),
}


def _freqs(R):
    return vdf.rope_frequencies(R, base=1000.0)[0]


def _positions(kind, B, N, gen):
    if kind == "none":
        return None
    if kind == "far":
        return (torch.randint(0, 1 << 30, (B, 1), generator=gen) + torch.arange(N)).cuda()
    if kind == "int32":
        return torch.randint(-5000, 5000, (N,), generator=gen, dtype=torch.int32).cuda()
    return (torch.rand((B, N), generator=gen) * 200 - 100).cuda()


def _heads(shape, dtype, gen, spread=1.0):
    B, N, H, D, _ = shape
    return (torch.randn((B, N, H, D), generator=gen) * spread + torch.randn(D, generator=gen) * 0.5).to(dtype).cuda()


@pytest.mark.parametrize("name", sorted(SHAPES))
@LAYOUTS
@TYPES
def test_shapes(name, layout, dtype):
    """The rotation, the norm with it and its gradients."""
    shape = SHAPES[name]
    say(f"[rope] {name} {shape} {layout} {dtype}")
    gen = torch.Generator().manual_seed(200 + sorted(SHAPES).index(name))
    B, N, H, D, R = shape
    x, g, f = _heads(shape, dtype, gen), _heads(shape, dtype, gen), _freqs(R)
    k, gk = _heads((B, N, max(1, H // 2), D, R), dtype, gen), _heads((B, N, max(1, H // 2), D, R), dtype, gen)
    pos = _positions("float", B, N, gen)
    w, wk = ((torch.rand(D, generator=gen) + 0.5).cuda() for _ in range(2))
    y = vdf.rope_forward(x, f, pos, layout)
    back = vdf.rope_forward(x, f, pos, layout, inverse=True)
    qn, kn = vdf.rope_norm_forward(x, k, w, wk, f, pos, pos, EPS, layout)
    grads = vdf.rope_norm_backward(x, k, g, gk, w, wk, f, pos, pos, EPS, layout)
    torch.cuda.synchronize()
    for got, inverse in ((y, False), (back, True)):
        want, mag = rotate(x, f, pos, layout, inverse=inverse)
        check("rotated", got, want, rounded(8 * U * mag, want, dtype))
        assert torch.equal(got[..., R:], x[..., R:])
    check("q", qn, *norm_rotate(x, w, f, pos, layout, EPS))
    check("k", kn, *norm_rotate(k, wk, f, pos, layout, EPS))
    (dq, tq), (dw, tw) = norm_rotate_grad(x, w, g, f, pos, layout, EPS)
    check("grad_q", grads[0], dq, tq)
    check("grad_q_weight", grads[2], dw, tw)
    (dk, tk), (dw, tw) = norm_rotate_grad(k, wk, gk, f, pos, layout, EPS)
    check("grad_k", grads[1], dk, tk)
    check("grad_k_weight", grads[3], dw, tw)


@pytest.mark.parametrize("kind", ["none", "far", "int32", "float"])
@LAYOUTS
def test_positions(kind, layout):
    """Indices, int64 past 2^30, negative int32 shared by the batch, coordinates."""
    gen = torch.Generator().manual_seed(230)
    shape = (3, 50, 2, 64, 64)
    x, f, pos = _heads(shape, F32, gen), _freqs(64), _positions(kind, 3, 50, gen)
    y = vdf.rope_forward(x, f, pos, layout)
    torch.cuda.synchronize()
    want, mag = rotate(x, f, pos, layout)
    check("rotated", y, want, 8 * U * mag)


def test_turns_are_exact_to_a_unit():
    """x = (1, 0) comes out as cosine and sine themselves: quarter turns, tiny and huge angles."""
    pos = torch.tensor([0.0, 1.0, -1.0, 2.0 ** -20, 0.25, 0.7853982, 1.5707964, 3.1415927, 4.712389,
                        6.2831855, 1e5, -1e7, 3e9, 1e12], device="cuda")
    x = torch.zeros((1, len(pos), 1, 2), device="cuda")
    x[..., 0] = 1
    y = vdf.rope_forward(x, torch.ones(1, dtype=torch.float64, device="cuda"), pos)
    torch.cuda.synchronize()
    t = pos.cpu().double()
    # the angle's place within a turn is off by 2^-52 of the angle
    slack = t.abs() * 2.0 ** -51
    check("cos", y[0, :, 0, 0], torch.cos(t), 3 * U * torch.cos(t).abs() + slack + 2.0 ** -30)
    check("sin", y[0, :, 0, 1], torch.sin(t), 3 * U * torch.sin(t).abs() + slack + 2.0 ** -30)


def test_turns_at_their_own_size():
    """Cosines and sines of angles from 2^-20 to 2^47, and next to quarter turns, where one of the two is
    small, by their own size.  The rest is exact to far below u = 2^-24 and rounds once to binary32 (its
    share of a sine is at most u, of a cosine pi / 4 u); the first term left out is 2^-27.7 of the result;
    the last multiply-add of a sine rounds by u, what it adds to y is at most a ninth of it and off by
    3 u: 2.5 u; the cosine's adds at most 0.41 of the result, off by 3 u too: 3.1 u and 0.1."""
    gen = torch.Generator().manual_seed(246)
    t = torch.exp2(torch.rand(6000, generator=gen) * 67 - 20) * (torch.randint(0, 2, (6000,), generator=gen) * 2 - 1)
    near = (torch.arange(1, 2000).double() * math.pi / 2).float()
    t = torch.cat([t, near, near * 4096, -near])
    x = torch.zeros((1, len(t), 2, 2), device="cuda")
    x[..., 0, 0], x[..., 1, 1] = 1, 1
    y = vdf.rope_forward(x, torch.ones(1, dtype=torch.float64, device="cuda"), t.cuda())
    torch.cuda.synchronize()
    c, s = (torch.tensor([f(v) for v in t.double().tolist()], dtype=torch.float64) for f in (math.cos, math.sin))
    tol = 3.2 * U
    check("cos", y[0, :, 0, 0], c, tol * c.abs())
    check("sin", y[0, :, 0, 1], s, tol * s.abs())
    check("-sin", y[0, :, 1, 0], -s, tol * s.abs())
    check("cos", y[0, :, 1, 1], c, tol * c.abs())


@LAYOUTS
def test_rotation_by_its_own_terms(layout):
    """y_a = x_a c - x_b s and y_b within their terms' own roundings: a turn's, 3.2 u of either, a product's
    and a multiply-add's, u each: 5.2 u of |x_a c| + |x_b s|, whatever the sizes beside each other."""
    gen = torch.Generator().manual_seed(247)
    x = torch.randn((2, 300, 3, 64), generator=gen) * torch.exp2(torch.randint(-12, 13, (2, 300, 3, 64), generator=gen))
    pos = torch.randint(0, 1 << 30, (2, 300), generator=gen)
    f = _freqs(64)
    y = vdf.rope_forward(x.cuda(), f, pos.cuda(), layout).cpu().double()
    t = pos.double()[..., None, None] * f.cpu()
    c, s, d = torch.cos(t), torch.sin(t), x.double()
    a, b = (d[..., ::2], d[..., 1::2]) if layout == "interleaved" else (d[..., :32], d[..., 32:])
    ya, yb = (y[..., ::2], y[..., 1::2]) if layout == "interleaved" else (y[..., :32], y[..., 32:])
    check("y_a", ya, a * c - b * s, 5.2 * U * ((a * c).abs() + (b * s).abs()))
    check("y_b", yb, b * c + a * s, 5.2 * U * ((b * c).abs() + (a * s).abs()))


def test_positions_that_are_no_numbers():
    """An infinite or NaN position makes its own token's rotated numbers NaN, no others."""
    gen = torch.Generator().manual_seed(231)
    x = _heads((1, 4, 3, 32, 16), F32, gen)
    pos = torch.tensor([1.0, math.inf, math.nan, 2.0], device="cuda")
    y = vdf.rope_forward(x, _freqs(16), pos)
    torch.cuda.synchronize()
    assert y[0, 1:3, :, :16].isnan().all() and torch.equal(y[..., 16:], x[..., 16:])
    assert y[0, [0, 3]].isfinite().all()


def test_angles_without_a_place_in_a_turn():
    """Pairs whose angles pass 2^52 are NaN, slower ones of the same token and the largest below are
    not: a position of 2^51 at frequencies 1, 2 and 2^-20."""
    x = _heads((1, 3, 2, 6, 6), F32, torch.Generator().manual_seed(243))
    f = torch.tensor([1.0, 2.0, 2.0 ** -20], dtype=torch.float64, device="cuda")
    pos = torch.tensor([2.0 ** 51, 3.0, -2.0 ** 51], device="cuda")
    y = vdf.rope_forward(x, f, pos, "interleaved")
    torch.cuda.synchronize()
    assert y[0, ::2, :, 2:4].isnan().all()
    assert y[0, ::2, :, [0, 1, 4, 5]].isfinite().all() and y[0, 1].isfinite().all()
    want, mag = rotate(x, f, pos.cpu(), "interleaved")
    keep = torch.ones_like(want, dtype=torch.bool)
    keep[0, ::2, :, 2:4] = False
    check("y", y.cpu()[keep], want[keep], (8 * U * mag)[keep])


@LAYOUTS
@TYPES
def test_what_is_not_rotated_stays(layout, dtype):
    """NaN and infinities past R reach no neighbour, and those numbers come out bit for bit."""
    gen = torch.Generator().manual_seed(232)
    x = _heads((2, 9, 3, 24, 10), dtype, gen)
    x[..., 11::2] = math.nan
    x[..., 10::4] = math.inf
    y = vdf.rope_forward(x, _freqs(10), None, layout)
    torch.cuda.synchronize()
    bits = torch.int32 if dtype == F32 else torch.int16
    assert y[..., :10].isfinite().all()
    assert torch.equal(y[..., 10:].view(bits), x[..., 10:].view(bits))


@TYPES
def test_views_and_in_place(dtype):
    """Views of a packed projection, read and written in place, off alignment; borders stay."""
    gen = torch.Generator().manual_seed(233)
    B, N, H, D = 2, 21, 4, 32
    f, pos = _freqs(D), _positions("far", B, N, gen)
    w, wk = ((torch.rand(D, generator=gen) + 0.5).cuda() for _ in range(2))
    packed = torch.randn((B, N, 3, H, D), generator=gen).to(dtype).cuda()
    first = packed.clone()
    q, k, v = packed.unbind(2)
    want = [norm_rotate(t, u, f, pos, "half", EPS) for t, u in ((q, w), (k, wk))]
    a, b = vdf.rope_norm_forward(q, k, w, wk, f, pos, pos, EPS)
    vdf.rope_norm_forward(q, k, w, wk, f, pos, pos, EPS, q_out=q, k_out=k)
    torch.cuda.synchronize()
    check("q", q, *want[0])
    check("k", k, *want[1])
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, first[:, :, 2])
    odd = torch.randn((B, N, H, D + 1), generator=gen).to(dtype).cuda()
    before = odd.clone()
    x = odd[..., 1:]
    want, mag = rotate(x, f, pos, "half")
    vdf.rope_forward(x, f, pos, out=x)
    torch.cuda.synchronize()
    check("x", x, want, rounded(8 * U * mag, want, dtype))
    assert torch.equal(odd[..., 0], before[..., 0])
    heads_first = torch.randn((B, H, N, D), generator=gen).to(dtype).cuda()
    y = vdf.rope_forward(heads_first.transpose(1, 2), f, pos)
    torch.cuda.synchronize()
    want, mag = rotate(heads_first.transpose(1, 2), f, pos, "half")
    check("y", y, want, rounded(8 * U * mag, want, dtype))
    with pytest.raises(vdf._lib.DAError, match="overlap"):
        vdf.rope_forward(x, f, pos, out=x.transpose(0, 0)[:1].expand(B, -1, -1, -1))
    with pytest.raises(vdf._lib.DAError, match="overlaps"):
        vdf.rope_norm_forward(q, k, w, wk, f, q_out=k, k_out=q)


@TYPES
def test_result_beside_its_input_in_one_buffer(dtype):
    """The second part of a packed tensor is the first one rotated, tokens or heads first."""
    gen = torch.Generator().manual_seed(245)
    B, N, H, D = 2, 21, 4, 32
    f = _freqs(D)
    for dim in (2, 1):
        packed = torch.randn((B, N, 2 * H, D) if dim == 2 else (B, 2 * H, N, D), generator=gen).to(dtype).cuda()
        before = packed.clone()
        x, y = (t if dim == 2 else t.transpose(1, 2) for t in packed.split(H, dim))
        vdf.rope_forward(x, f, out=y)
        torch.cuda.synchronize()
        want, mag = rotate(x, f, None, "half")
        check("y", y, want, rounded(8 * U * mag, want, dtype))
        assert torch.equal(packed.split(H, dim)[0], before.split(H, dim)[0])
        with pytest.raises(vdf._lib.DAError, match="overlaps"):
            vdf.rope_forward(x[..., :16], f[:8], out=x[..., 8:24])


def test_magnitude_and_scaled_frequencies():
    gen = torch.Generator().manual_seed(234)
    x = _heads((2, 40, 3, 64, 64), F32, gen)
    for scaling in ("linear", "base", "blend"):
        f, m = vdf.rope_frequencies(64, scaling=scaling, factor=8.0, trained=512)
        pos = torch.arange(40, device="cuda") * 100
        y = vdf.rope_forward(x, f, pos, "half", m)
        torch.cuda.synchronize()
        want, mag = rotate(x, f, pos, "half", m)
        check(scaling, y, want, 8 * U * mag)


@TYPES
def test_norm_of_different_sides(dtype):
    """k of other batch, tokens and heads than q, or none, without weights."""
    gen = torch.Generator().manual_seed(235)
    q, k = _heads((2, 30, 4, 48, 48), dtype, gen), _heads((3, 7, 2, 48, 48), dtype, gen)
    f = _freqs(48)
    qp, kp = _positions("float", 2, 30, gen), _positions("int32", 3, 7, gen)
    w = (torch.rand(48, generator=gen) + 0.5).cuda()
    a, b = vdf.rope_norm_forward(q, k, None, w, f, qp, kp, EPS, "interleaved")
    c, none = vdf.rope_norm_forward(q, None, None, None, f, qp, None, EPS, "interleaved")
    torch.cuda.synchronize()
    check("q", a, *norm_rotate(q, None, f, qp, "interleaved", EPS))
    check("k", b, *norm_rotate(k, w, f, kp, "interleaved", EPS))
    assert torch.equal(a, c) and none is None
    g = _heads((2, 30, 4, 48, 48), dtype, gen)
    dq, dk, dw, dkw = vdf.rope_norm_backward(q, None, g, None, None, None, f, qp, None, EPS, "interleaved")
    torch.cuda.synchronize()
    (want, tol), (ww, tw) = norm_rotate_grad(q, None, g, f, qp, "interleaved", EPS)
    check("grad_q", dq, want, tol)
    check("grad_q_weight", dw, ww, tw)
    assert dk is None and dkw is None


def test_no_tokens():
    f = _freqs(16)
    x = torch.empty((2, 0, 3, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    assert vdf.rope_forward(x, f).shape == x.shape
    dq, dk, dw, dkw = vdf.rope_norm_backward(x, x, x, x, w, w, f)
    torch.cuda.synchronize()
    assert dq.shape == x.shape and (dw == 0).all() and (dkw == 0).all()
    y = torch.randn((1, 4, 3, 16), device="cuda")
    dq, dk, dw, dkw = vdf.rope_norm_backward(x, y, x, y, w, w, f)
    torch.cuda.synchronize()
    (_, _), (want, tol) = norm_rotate_grad(y, w, y, f, None, "half", EPS)
    check("grad_k_weight", dkw, want, tol)
    assert (dw == 0).all()


def test_weight_gradients_of_many_rows():
    """200000 rows: the workgroups' sums join in binary64.  A lane adds up fewer than 200 rows of
    them, so 250 u of the magnitudes hold."""
    gen = torch.Generator().manual_seed(236)
    shape = (2, 12500, 8, 32, 32)
    x, g, f = _heads(shape, F32, gen), _heads(shape, F32, gen), _freqs(32)
    w = torch.ones(32, device="cuda")
    _, _, dw, _ = vdf.rope_norm_backward(x, None, g, None, w, None, f)
    torch.cuda.synchronize()
    _, (want, tol) = norm_rotate_grad(x, w, g, f, None, "half", EPS)
    check("grad_weight", dw, want, tol * 250 / 200000)


def test_large_and_small_rows():
    """Rows of 1e-18, 1e18 and zeros: squares within binary32, eps beside them."""
    gen = torch.Generator().manual_seed(237)
    x = torch.randn((1, 4, 2, 64), generator=gen)
    x[:, 0] *= 1e-18
    x[:, 1] *= 1e18
    x[:, 2] = 0
    x, f = x.cuda(), _freqs(64)
    y, _ = vdf.rope_norm_forward(x, None, None, None, f, eps=1e-6)
    torch.cuda.synchronize()
    check("y", y, *norm_rotate(x, None, f, None, "half", 1e-6))
    assert (y[0, 2] == 0).all()


def test_every_half_precision_rounding_is_once():
    gen = torch.Generator().manual_seed(238)
    for dt in (BF16, F16):
        x = _heads((2, 33, 3, 64, 64), dt, gen)
        full = vdf.rope_norm_forward(x.float(), None, None, None, _freqs(64))[0]
        got = vdf.rope_norm_forward(x, None, None, None, _freqs(64))[0]
        torch.cuda.synchronize()
        # 32-bit results differ by the order of a sum alone
        assert ((got.double() - full.double()).abs() <= full.double().abs() * (HALF[dt] + 80 * U)).all()


@pytest.mark.parametrize("dtype, wdtype", [(F32, F32), (BF16, F32), (F16, F16)])
@LAYOUTS
def test_autograd(dtype, wdtype, layout):
    gen = torch.Generator().manual_seed(239)
    shape = (2, 25, 4, 32, 16)
    q, k = _heads(shape, dtype, gen).requires_grad_(True), _heads((2, 9, 2, 32, 16), dtype, gen).requires_grad_(True)
    w, wk = ((torch.rand(32, generator=gen) + 0.5).cuda().to(wdtype).requires_grad_(True) for _ in range(2))
    g, gk = _heads(shape, dtype, gen), _heads((2, 9, 2, 32, 16), dtype, gen)
    f, pos = _freqs(16), _positions("float", 2, 25, gen)
    a, b = vdf.norm_rotary(q, k, w, wk, f, pos, None, EPS, layout)
    ((a.float() * g.float()).sum() + (b.float() * gk.float()).sum()).backward()
    torch.cuda.synchronize()
    for x, ww, gg, p in ((q, w, g, pos), (k, wk, gk, None)):
        (dx, tx), (dw, tw) = norm_rotate_grad(x, ww.float(), gg, f, p, layout, EPS)
        check("x.grad", x.grad, dx, tx)
        check("w.grad", ww.grad, dw, rounded(tw, dw, wdtype))
        assert x.grad.dtype == dtype and ww.grad.dtype == wdtype
    x = _heads(shape, dtype, gen).requires_grad_(True)
    (vdf.rotary(x, f, pos, layout, 1.5).float() * g.float()).sum().backward()
    torch.cuda.synchronize()
    want, mag = rotate(g, f, pos, layout, 1.5, inverse=True)
    check("x.grad", x.grad, want, rounded(8 * U * mag, want, dtype))


@pytest.mark.parametrize("need", ["all", "weights", "k_weight"])
def test_autograd_without_keys(need):
    """k None, its weight a leaf all the same, as a module that holds both passes it: its gradient is
    none, the others are those of the queries alone."""
    gen = torch.Generator().manual_seed(244)
    shape = (2, 25, 4, 32, 16)
    q, g = _heads(shape, F32, gen), _heads(shape, F32, gen)
    w, wk = ((torch.rand(32, generator=gen) + 0.5).cuda().requires_grad_(need != "k_weight" or n == 1)
             for n in range(2))
    q.requires_grad_(need == "all" or need == "k_weight")
    f = _freqs(16)
    y, none = vdf.norm_rotary(q, None, w, wk, f, None, None, EPS)
    assert none is None
    y.backward(g)
    torch.cuda.synchronize()
    (dx, tx), (dw, tw) = norm_rotate_grad(q, w, g, f, None, "half", EPS)
    assert wk.grad is None
    if q.requires_grad:
        check("q.grad", q.grad, dx, tx)
    if w.requires_grad:
        check("w.grad", w.grad, dw, tw)


def test_gradient_against_differences():
    """Along the gradient, the norm's own forward: a step of h = 2^-8 of unit length moves a row of
    root mean square near 1 by a third derivative of a few times the gradient's size."""
    gen = torch.Generator().manual_seed(240)
    x, g = _heads((1, 6, 2, 16, 16), F32, gen), _heads((1, 6, 2, 16, 16), F32, gen)
    w, f = (torch.rand(16, generator=gen) + 0.5).cuda(), _freqs(16)
    dx, _, dw, _ = vdf.rope_norm_backward(x, None, g, None, w, None, f)
    h = 2.0 ** -8

    def loss(xx, ww):
        return (vdf.rope_norm_forward(xx, None, ww, None, f)[0].double() * g.double()).sum()

    t = dx / dx.norm()
    want = (loss(x + h * t, w) - loss(x - h * t, w)) / (2 * h)
    rounding = 2.0 ** -19 * float(g.abs().sum()) / h
    assert abs(float(want - dx.double().norm())) <= 16 * h * h * float(dx.norm()) + rounding
    t = dw / dw.norm()
    want = (loss(x, w + h * t) - loss(x, w - h * t)) / (2 * h)
    assert abs(float(want - dw.double().norm())) <= rounding


def test_graph_replays_match_eager():
    gen = torch.Generator().manual_seed(241)
    shape = (2, 300, 6, 64, 64)
    q, g = _heads(shape, BF16, gen), _heads(shape, BF16, gen)
    k, gk = _heads((2, 300, 2, 64, 64), BF16, gen), _heads((2, 300, 2, 64, 64), BF16, gen)
    w, f = (torch.rand(64, generator=gen) + 0.5).cuda(), _freqs(64)
    pos = _positions("far", 2, 300, gen)
    ws = torch.empty(vdf.rope_norm_backward_workspace_size(q, k), dtype=torch.uint8, device="cuda")

    def step():
        return (*vdf.rope_norm_forward(q, k, w, w, f, pos, pos),
                *vdf.rope_norm_backward(q, k, g, gk, w, w, f, pos, pos, workspace=ws),
                vdf.rope_forward(q, f, pos))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(4):
        pos.add_(17)
        q.mul_(1.25)
        ws.fill_(0xff)
        for t in got:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {n}"


def test_more_numbers_than_32_bits_count():
    """2 x 600000 tokens x 32 heads x 128 bfloat16 numbers: tokens around place 2^32."""
    B, N, H, D = 2, 600000, 32, 128
    x = torch.empty((B, N, H, D), dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(242)
    for b in range(B):
        for r in range(0, N, 50000):
            x[b, r:r + 50000] = torch.randn((50000, H, D), generator=gen, device="cuda", dtype=BF16)
    f = _freqs(D)
    edge = 2 ** 32 // (H * D) - N
    rows = [(0, 0), (1, edge - 3), (1, N - 6)]
    parts = [x[b:b + 1, n:n + 6].clone() for b, n in rows]
    w = torch.rand(D, device="cuda") + 0.5
    vdf.rope_norm_forward(x, None, w, None, f, q_out=x)
    torch.cuda.synchronize()
    for (b, n), part in zip(rows, parts):
        pos = torch.arange(n, n + 6)
        check("y", x[b:b + 1, n:n + 6], *norm_rotate(part, w, f, pos, "half", EPS))


def test_refusals_on_the_gpu():
    x, f = torch.zeros((2, 3, 4, 8), device="cuda"), _freqs(8)
    with pytest.raises(ValueError, match="layout"):
        vdf.rope_forward(x, f, layout="quarter")
    with pytest.raises(TypeError, match="positions"):
        vdf.rope_forward(x, f, torch.zeros(3, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError, match="positions"):
        vdf.rope_forward(x, f, torch.zeros((3, 3), device="cuda"))
    with pytest.raises(TypeError, match="freqs"):
        vdf.rope_forward(x, f.float())
    with pytest.raises(vdf._lib.DAError, match="rotated"):
        vdf.rope_forward(x, _freqs(10))
    with pytest.raises(ValueError, match="out"):
        vdf.rope_forward(x, f, out=x[:1])
    with pytest.raises(ValueError, match="q_weight"):
        vdf.rope_norm_forward(x, None, torch.ones(7, device="cuda"), None, f)
