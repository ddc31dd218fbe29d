"""Group norm with an activation, forward and backward, on the GPU against the definition in
64 bits (norm_int8_reference.py has the bounds and how they come about): group widths that
divide a 16-byte vector, straddle one and pass a workgroup; one row and many; types and
activations; large means and outliers; NaNs; views off alignment; in place; streams, graphs
and autograd."""
import itertools

import pytest
import torch

import view_deformable_feature_amd as vdf
from gpu_helpers import say
from norm_int8_reference import HALF, U, Norm, act_grad, check, gelu_tols, rounded

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5

# N, S, C, G
SHAPES = {
    "vector_in_group": (2, 35, 64, 4),
    "group_is_channel": (2, 19, 24, 24),
    "two_groups_a_vector": (3, 33, 64, 16),         # 4 channels: half a 16-bit vector
    "groups_of_three": (2, 17, 48, 16),             # straddle vectors of any type
    "groups_of_six": (1, 50, 96, 16),
    "odd_channels": (2, 23, 21, 3),                 # no vectors
    "one_channel": (2, 9, 1, 1),
    "one_row": (3, 1, 64, 2),
    "two_rows": (1, 2, 256, 8),
    "one_group": (2, 40, 512, 1),
    "wide_group": (1, 7, 4096, 1),                  # cut into units, with vectors
    "wide_ragged_group": (1, 5, 5200, 2),           # the last unit shorter
    "wide_odd_group": (2, 6, 8 * 257, 8),           # cut into units, no vectors
    "ragged_slabs": (1, 37, 320, 5),
    "many_chunks": (1, 30011, 8, 2),
    "images": (37, 11, 32, 4),
    "level_8x22": (6, 176, 256, 8),
    "stage_28x28": (3, 784, 256, 32),
    "level_64x176": (1, 11264, 256, 32),
    "stage_56x56": (4, 3136, 128, 32),
    # slabs of less than 64 bytes of a row: the most rows (forward 4096, backward 2048), one more
    "narrow_2048": (1, 2048, 64, 8),
    "narrow_2049": (1, 2049, 64, 8),
    "narrow_4096": (2, 4096, 64, 8),
    "narrow_4097": (2, 4097, 64, 8),
}


def _inputs(shape, dtype, seed, dy_dtype=None):
    N, S, C, G = shape
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((N, S, C), generator=gen) * (torch.rand((C,), generator=gen) * 1.5 + 0.5)
    x = (x + torch.randn((C,), generator=gen) * 0.5 + 0.4).to(dtype)
    w = torch.rand((C,), generator=gen) + 0.5
    w[::3] *= -1
    b = torch.randn((C,), generator=gen) * 0.3
    dy = torch.randn((N, S, C), generator=gen).to(dy_dtype or dtype)
    return tuple(t.cuda() for t in (x, w, b, dy))


def _check(shape, dtype, name, out_dtype=None, seed=1, params=True, x=None):
    G = shape[3]
    odt = out_dtype or dtype
    ix, w, b, dy = _inputs(shape, dtype, seed, odt)
    x = ix if x is None else x
    if not params:
        w = b = None
    out, mean, rstd = vdf.gn_forward(x, G, w, b, EPS, name, out_dtype=out_dtype)
    grads = vdf.gn_backward(x, dy, mean, rstd, G, w, b, name)
    torch.cuda.synchronize()
    ref = Norm(x, G, w, b, EPS, name)
    assert out.dtype == odt and grads[0].dtype == dtype
    tm, tr = ref.stat_tols()
    check("mean", mean, ref.mean, tm)
    check("rstd", rstd, ref.rstd, tr)
    check("out", out, ref.y, ref.out_tol(odt))
    (dx, dw, db), (tx, tw, tb) = ref.backward(dy)
    check("grad_weight", grads[1], dw, tw)
    check("grad_bias", grads[2], db, tb)
    check("grad_x", grads[0], dx, rounded(tx, dx, dtype))
    return x, w, b, dy, out, mean, rstd, grads


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_shapes(name, dtype):
    say(f"[gn] {name} {SHAPES[name]} {dtype}")
    _check(SHAPES[name], dtype, "silu", seed=10 + sorted(SHAPES).index(name))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("params", [True, False], ids=["affine", "plain"])
def test_activations(act, params):
    _check((2, 61, 64, 8), F32, act, seed=31, params=params)
    _check((2, 61, 64, 8), BF16, act, seed=32, params=params)


@pytest.mark.parametrize("x_dtype, out_dtype", list(itertools.product([F32, BF16, F16], repeat=2)))
def test_types(x_dtype, out_dtype):
    _check((2, 29, 96, 6), x_dtype, "gelu", out_dtype=out_dtype, seed=41)
    _check((2, 29, 33, 3), x_dtype, "relu", out_dtype=out_dtype, seed=42)


@pytest.mark.parametrize("offset", [1e3, -2e4])
def test_large_mean(offset):
    """A common offset that the squares would drown in."""
    x, _, _, _ = _inputs((2, 300, 32, 4), F32, 51)
    _check((2, 300, 32, 4), F32, "none", seed=51, x=x + offset)


def test_outlier_in_the_first_row():
    """The row that deviations are taken from is far from all others."""
    shape = (1, 3000, 32, 4)
    x, _, _, _ = _inputs(shape, F32, 52)
    x = x.clone()
    x[:, 0] *= 60
    x[:, 0, :8] = 3e3
    _check(shape, F32, "silu", seed=52, x=x)


def test_constant_groups():
    """No spread: the variance is exactly 0, the result is the bias."""
    shape = (2, 21, 32, 4)
    _, w, b, dy = _inputs(shape, F32, 53)
    x = torch.full((2, 21, 32), 7.25, device="cuda")
    out, mean, rstd = vdf.gn_forward(x, 4, w, b, EPS)
    torch.cuda.synchronize()
    assert torch.equal(mean, torch.full_like(mean, 7.25))
    assert torch.equal(out, b.expand_as(out))
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_bad_values_stay_in_their_group(bad):
    shape = (3, 40, 64, 8)
    x, w, b, dy = _inputs(shape, F32, 54)
    x = x.clone()
    x[1, 17, 5 * 8 + 3] = bad
    out, mean, rstd = vdf.gn_forward(x, 8, w, b, EPS, "relu")
    gx, _, _ = vdf.gn_backward(x, dy, mean, rstd, 8, w, b, "relu")
    torch.cuda.synchronize()
    hit = torch.zeros((3, 40, 64), dtype=torch.bool, device="cuda")
    hit[1, :, 40:48] = True
    assert out[hit].isnan().all() and not out[~hit].isnan().any()
    assert gx[hit].isnan().all() and not gx[~hit].isnan().any()
    assert rstd[1, 5].isnan() and int(rstd.isnan().sum()) == 1


def test_eps_zero_and_large():
    shape = (2, 30, 16, 2)
    x, w, b, _ = _inputs(shape, F32, 55)
    for eps in (0.0, 10.0):
        out, _, rstd = vdf.gn_forward(x, 2, w, b, eps)
        torch.cuda.synchronize()
        ref = Norm(x, 2, w, b, eps, "none")
        check("rstd", rstd, ref.rstd, ref.stat_tols()[1])
        check("out", out, ref.y, ref.out_tol(F32))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_views_off_alignment(dtype):
    """x, grad_out and out one element into larger buffers: no vectors, the same numbers
    within the bounds."""
    shape = (2, 45, 64, 4)
    x, w, b, dy = _inputs(shape, dtype, 56)

    def shifted(t):
        v = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:].view(t.shape)
        v.copy_(t)
        return v

    xs, dys, outs, gxs = shifted(x), shifted(dy), shifted(x), shifted(x)
    assert xs.data_ptr() % 16
    ref = Norm(x, 4, w, b, EPS, "silu")
    (dx, _, _), (tx, _, _) = ref.backward(dy)
    for xi, di, oi, gi in ((xs, dys, outs, gxs), (x, dy, outs, gxs), (xs, dy, None, None)):
        out, mean, rstd = vdf.gn_forward(xi, 4, w, b, EPS, "silu", out=oi)
        gx, _, _ = vdf.gn_backward(xi, di, mean, rstd, 4, w, b, "silu", grad_x=gi)
        torch.cuda.synchronize()
        check("out", out, ref.y, ref.out_tol(dtype))
        check("grad_x", gx, dx, rounded(tx, dx, dtype))


@pytest.mark.parametrize("shape", [(2, 33, 64, 4), (2, 5000, 64, 4), (1, 9, 21, 3),
                                   (4, 40000, 64, 8), (1, 30011, 4096, 1)])
def test_in_place(shape):
    x, w, b, dy = _inputs(shape, BF16, 57)
    out, mean, rstd = vdf.gn_forward(x, shape[3], w, b, EPS, "silu")
    gx, gw, gb = vdf.gn_backward(x, dy, mean, rstd, shape[3], w, b, "silu")
    x2, dy2 = x.clone(), dy.clone()
    vdf.gn_forward(x2, shape[3], w, b, EPS, "silu", out=x2)
    gx2, gw2, gb2 = vdf.gn_backward(x, dy2, mean, rstd, shape[3], w, b, "silu", grad_x=dy2)
    torch.cuda.synchronize()
    assert torch.equal(x2, out) and torch.equal(gx2, gx)
    assert torch.equal(gw2, gw) and torch.equal(gb2, gb)


def test_image_dimensions_and_parts():
    """[N, H, W, C] maps are [N, H * W, C]; parts that nobody asks for are left out."""
    x, w, b, dy = _inputs((2, 35, 32, 4), F32, 58)
    out, mean, rstd = vdf.gn_forward(x, 4, w, b, EPS, "silu")
    o4, _, _ = vdf.gn_forward(x.view(2, 5, 7, 32), 4, w, b, EPS, "silu")
    gx, gw, gb = vdf.gn_backward(x, dy, mean, rstd, 4, w, b, "silu")
    only_x = vdf.gn_backward(x, dy, mean, rstd, 4, w, b, "silu", need_params=False)
    only_p = vdf.gn_backward(x, dy, mean, rstd, 4, w, b, "silu", need_x=False)
    torch.cuda.synchronize()
    assert o4.shape == (2, 5, 7, 32) and torch.equal(o4.view_as(out), out)
    assert torch.equal(only_x[0], gx) and only_x[1] is None and only_x[2] is None
    assert only_p[0] is None and torch.equal(only_p[1], gw) and torch.equal(only_p[2], gb)


def test_empty_batch():
    x = torch.zeros((0, 5, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    out, mean, rstd = vdf.gn_forward(x, 4, w, w)
    gx, gw, gb = vdf.gn_backward(x, x, mean, rstd, 4, w, w)
    torch.cuda.synchronize()
    assert out.shape == x.shape and mean.shape == (0, 4) and gx.shape == x.shape
    assert torch.equal(gw, torch.zeros_like(w)) and torch.equal(gb, torch.zeros_like(w))


def test_repeatable():
    x, w, b, dy = _inputs((4, 3001, 96, 12), BF16, 59)
    runs = []
    for _ in range(2):
        out, mean, rstd = vdf.gn_forward(x, 12, w, b, EPS, "silu")
        runs.append((out, mean, rstd) + vdf.gn_backward(x, dy, mean, rstd, 12, w, b, "silu"))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*runs))


def test_another_stream():
    """The work goes to the current stream, its workspace too."""
    x, w, b, dy = _inputs((8, 4000, 64, 8), F32, 60)
    want = vdf.gn_forward(x, 8, w, b, EPS, "silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = vdf.gn_forward(x, 8, w, b, EPS, "silu")
        g1 = vdf.gn_backward(x, dy, a[1], a[2], 8, w, b, "silu")
    c = vdf.gn_forward(x, 8, w, b, EPS, "silu")
    g2 = vdf.gn_backward(x, dy, want[1], want[2], 8, w, b, "silu")
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, a))
    assert all(torch.equal(p, q) for p, q in zip(want, c))
    assert all(torch.equal(p, q) for p, q in zip(g1, g2))


@pytest.mark.parametrize("shape, dtype", [((8, 784, 64, 8), BF16), ((2, 20000, 64, 8), F32)])
def test_graph_replays_match_eager(shape, dtype):
    """A forward and a backward captured and replayed, eager work on the same buffers
    between the replays."""
    G = shape[3]
    x, w, b, dy = _inputs(shape, dtype, 61)
    ws = torch.empty(max(1, vdf.gn_workspace_size(x, G)), device="cuda", dtype=torch.uint8)
    bws = torch.empty(max(1, vdf.gn_backward_workspace_size(x, G)), device="cuda", dtype=torch.uint8)

    def step():
        out, mean, rstd = vdf.gn_forward(x, G, w, b, EPS, "silu", workspace=ws)
        return (out, mean, rstd) + vdf.gn_backward(x, dy, mean, rstd, G, w, b, "silu", workspace=bws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    first = x.clone()
    for k in range(4):
        x.copy_(first).mul_(1 + 0.25 * k)
        ws.fill_(0xff)
        bws.fill_(0xff)
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), f"replay {k}"


@pytest.mark.parametrize("dtype, pdtype", [(F32, F32), (BF16, F32), (F16, F16), (BF16, BF16)])
def test_autograd(dtype, pdtype):
    shape = (2, 5, 9, 24)
    gen = torch.Generator().manual_seed(62)
    x = torch.randn(shape, generator=gen).cuda().to(dtype).requires_grad_(True)
    w = (torch.rand(24, generator=gen) + 0.5).cuda().to(pdtype).requires_grad_(True)
    b = torch.randn(24, generator=gen).cuda().to(pdtype).requires_grad_(True)
    dy = torch.randn(shape, generator=gen).cuda()
    out = vdf.group_norm_act(x, 3, w, b, EPS, "gelu", out_dtype=F32)
    (out * dy).sum().backward()
    torch.cuda.synchronize()
    ref = Norm(x.view(2, 45, 24), 3, w.float(), b.float(), EPS, "gelu")
    (dx, dw, db), (tx, tw, tb) = ref.backward(dy.view(2, 45, 24))
    assert x.grad.dtype == dtype and w.grad.dtype == pdtype
    check("x.grad", x.grad, dx, rounded(tx, dx, dtype))
    check("w.grad", w.grad, dw, rounded(tw, dw, pdtype))
    check("b.grad", b.grad, db, rounded(tb, db, pdtype))


def test_autograd_of_a_transposed_map_and_without_parameters():
    """A channels-first tensor seen as channels last is copied; no parameters, no
    gradients of them; a second derivative is refused."""
    x = torch.randn((2, 16, 6, 5), device="cuda", requires_grad=True)
    out = vdf.group_norm_act(x.permute(0, 2, 3, 1), 4, activation="silu")
    g, = torch.autograd.grad(out.sum(), x, create_graph=True)
    torch.cuda.synchronize()
    ref = Norm(x.permute(0, 2, 3, 1).reshape(2, 30, 16), 4, None, None, EPS, "silu")
    (dx, _, _), (tx, _, _) = ref.backward(torch.ones(2, 30, 16))
    check("x.grad", g.permute(0, 2, 3, 1).reshape(2, 30, 16), dx, tx)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradient_against_differences(act):
    """Central differences of the library's own forward, along the gradient itself: x moves by
    h = 2^-6, and the difference quotient of L = sum(y * dy) is off the gradient's length by
    h^2 / 6 times a third derivative (at most 320 max |dy| for a step of length 1 here) and by
    the rounding of y, 2^-18 sum |dy| / h: under 1 % of that length in all."""
    shape = (2, 24, 16, 2)
    x, w, b, dy = _inputs(shape, F32, 63)
    h = 2.0 ** -6

    def loss(xx):
        return (vdf.gn_forward(xx, 2, w, b, EPS, act)[0].double() * dy.double()).sum()

    _, mean, rstd = vdf.gn_forward(x, 2, w, b, EPS, act)
    gx, _, _ = vdf.gn_backward(x, dy, mean, rstd, 2, w, b, act)
    t = gx / gx.norm()
    want = (loss(x + h * t) - loss(x - h * t)) / (2 * h)
    got = (gx.double() * t.double()).sum()
    total = float(dy.double().abs().max()) * 32
    assert abs(float(got - want)) <= 10 * total * h * h / 6 + 2.0 ** -18 * float(dy.abs().sum()) / h


def test_every_half_precision_rounding_is_once():
    """A 16-bit result is the 32-bit one rounded to nearest even."""
    x, w, b, _ = _inputs((2, 77, 64, 4), F32, 65)
    full, _, _ = vdf.gn_forward(x, 4, w, b, EPS, "silu")
    for dt in (BF16, F16):
        got, _, _ = vdf.gn_forward(x, 4, w, b, EPS, "silu", out_dtype=dt)
        torch.cuda.synchronize()
        assert torch.equal(got, full.to(dt)) and HALF[dt]


def test_more_values_than_32_bits_count():
    """2 x 1100003 x 2048 bfloat16 values: places past 2^32 in the second image's rows."""
    N, S, C, G = 2, 1100003, 2048, 32
    x = torch.empty((N, S, C), device="cuda", dtype=BF16)
    gen = torch.Generator(device="cuda").manual_seed(70)
    for n in range(N):
        for r in range(0, S, 100000):
            part = x[n, r:r + 100000]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=BF16))
    w = torch.rand((C,), device="cuda") + 0.5
    out, mean, rstd = vdf.gn_forward(x, G, w, None, EPS, "relu")
    torch.cuda.synchronize()
    for n, r in ((0, 0), (1, 0), (1, S - 300)):
        rows = x[n, r:r + 300].double()
        z = ((rows.view(-1, G, C // G) - mean[n].double()[None, :, None])
             * rstd[n].double()[None, :, None]).view(-1, C) * w.double()
        want = z.clamp_min(0)
        got = out[n, r:r + 300].double()
        assert ((got - want).abs() <= 2.0 ** -8 * want + 1e-5).all()
    # the averages of 70 million normal numbers
    assert mean.abs().max() < 1e-3 and (rstd - 1).abs().max() < 1e-3
    gx, _, _ = vdf.gn_backward(x, out, mean, rstd, G, w, None, "none", need_params=False,
                               grad_x=out)
    torch.cuda.synchronize()
    assert gx[1, -1].isfinite().all() and gx[1, -1].abs().max() > 0


@pytest.mark.parametrize("shape, dtype", [((6, 176, 256, 8), F32), ((2, 784, 256, 32), BF16),
                                          ((1, 196, 512, 32), F16), ((2, 4095, 64, 8), F32)])
def test_mean_far_from_the_first_value(shape, dtype):
    """Each group's first value is 1000, all others are whole numbers below 8, constant along
    the rows.  Differences from the first value are whole numbers and a thread's sums of them are
    exact, but for the thread (at most 16 rows, 8 channels) that holds it: its mean of that
    channel is off by 2 u 1000, its sum over channels and that times its rows by u 8000 each.
    Joined in 64 bits and rounded once, the mean is off by u |mean| and that thread's share of the
    group; a join in 32 bits would round a number of the size of 1000."""
    N, S, C, G = shape
    x = (torch.arange(C) * 7 % 8).float().expand(N, S, C).clone()
    x[:, 0, ::C // G] = 1000.0
    x = x.to(dtype).cuda()
    _, mean, rstd = vdf.gn_forward(x, G, None, None, EPS)
    torch.cuda.synchronize()
    ref = Norm(x, G, None, None, EPS, "none")
    share = 18000.0 * 16 / (S * C // G)
    check("mean", mean, ref.mean, U * (ref.mean.abs() + share))
    check("rstd", rstd, ref.rstd, ref.stat_tols()[1])


def test_gelu_derivative_in_the_lower_tail():
    """z = x exactly (mean 0, rstd 1 given, one row): grad_bias is the derivative, by whole slabs
    and, with another type of grad_out, by chunks."""
    z = (torch.arange(256) - 128).float() / 16
    x, one = z.view(1, 1, 256).cuda(), torch.ones((1, 1), device="cuda")
    for dtype in (F32, BF16):
        dy = torch.ones((1, 1, 256), device="cuda", dtype=dtype)
        _, _, db = vdf.gn_backward(x, dy, 0 * one, one, 1, None, None, "gelu")
        torch.cuda.synchronize()
        check("grad_bias", db, act_grad(z.double(), "gelu"), gelu_tols(z.double())[1])


@pytest.mark.parametrize("dy_dtype", [F32, BF16], ids=["whole", "chunks"])
def test_parameter_gradients_of_many_images(dy_dtype):
    """5000 images, one of them with a gradient of 1 and the others with 0.9 u each, which vanish
    beside it where they are added one after the other in 32 bits.  Each image's own sum has one
    term that is not 0, so grad_bias is exact before its one rounding; grad_weight's terms are
    products of three rounded numbers, x - mean, rstd and the gradient."""
    N, S, C, G = 5000, 2, 16, 2
    x, _, _, _ = _inputs((N, S, C, G), F32, 66)
    dy = torch.zeros((N, S, C))
    dy[:, 0] = 0.8984375 * U
    dy[0, 0] = 1
    dy = dy.to(dy_dtype).cuda()
    _, mean, rstd = vdf.gn_forward(x, G, None, None, EPS)
    gx, dw, db = vdf.gn_backward(x, dy, mean, rstd, G)
    torch.cuda.synchronize()
    d = dy.cpu().double()
    check("grad_bias", db, d.sum((0, 1)), 1.001 * U * d.sum((0, 1)))
    per = C // G
    xhat = ((x.cpu().double().view(N, S, G, per) - mean.cpu().double()[:, None, :, None])
            * rstd.cpu().double()[:, None, :, None]).view(N, S, C)
    terms = d * xhat
    check("grad_weight", dw, terms.sum((0, 1)), 5 * U * terms.abs().sum((0, 1)))
    check("grad_x", gx, *_grad_x_of(x, dy, mean, rstd, G))


def _grad_x_of(x, dy, mean, rstd, G, w=None):
    """grad_x without an activation from the given statistics, in 64 bits, and its bound: the
    averages' terms and their sum over a thread's rows and channels round at most 32 times, the
    result a few times more."""
    N, S, C = x.shape

    def split(t):
        return t.double().reshape(N, S, G, C // G)

    r = rstd.double()[:, None, :, None]
    xhat = (split(x) - mean.double()[:, None, :, None]) * r
    wdz = split(dy.double() * (1 if w is None else w.double()))
    m1, m2 = wdz.mean((1, 3), keepdim=True), (wdz * xhat).mean((1, 3), keepdim=True)
    tol = 40 * U * r * (wdz.abs() + wdz.abs().mean((1, 3), keepdim=True)
                        + xhat.abs() * (wdz * xhat).abs().mean((1, 3), keepdim=True)) + 2.0 ** -149
    return ((r * (wdz - m1 - xhat * m2)).reshape(N, S, C).cpu(), tol.reshape(N, S, C).cpu())


# Slabs of several groups in one workgroup, which maps of more than 4 MB and many images get.
WIDE = {
    "stage_28x28_batch": (12, 784, 256, 32),        # 64 bytes of a row: 2 to 4 groups
    "stage_56x56_batch": (6, 3136, 128, 32),        # 16-bit forward: 8 groups, 13 vectors a thread
    "four_vectors_wide": (64, 400, 256, 32),        # 16-bit backward: 128 bytes, 8 groups
    "shorter_last_slab": (128, 200, 96, 3),         # 16-bit: slabs of 64 and 32 channels
    "shorter_last_odd_slab": (90, 100, 105, 7),     # no vectors: slabs of 30 and 15 channels
}


@pytest.mark.parametrize("name", sorted(WIDE))
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_wide_slabs(name, dtype):
    say(f"[gn] wide {name} {WIDE[name]} {dtype}")
    _check(WIDE[name], dtype, "gelu", seed=40 + sorted(WIDE).index(name))


@pytest.mark.parametrize("shape", [(2, 300, 64, 4), (1, 40000, 64, 4), (1, 7, 4096, 1)],
                         ids=["whole", "chunks", "units"])
def test_large_deviations(shape):
    """Deviations of up to 2^46, whose squares and their sums stay in binary32."""
    x, _, _, _ = _inputs(shape, F32, 67)
    x = x / x.abs().max() * 2.0 ** 46
    _check(shape, F32, "none", seed=67, x=x)


def test_gradients_of_more_values_than_32_bits_count():
    """2 x 1100003 x 2048 bfloat16 values: grad_x at rows of both images, around and past place
    2^32, and the parameters' gradients, against averages and sums formed in 64 bits by slices.
    Each image's gradient has a mean and a share of x of its own, so that the averages of the
    other image, or of other rows, would show.  A thread adds up 68 rows of 8 channels and a
    workgroup 16 of its rows before the sums meet in 64 bits: 100 u of the magnitudes."""
    N, S, C, G = 2, 1100003, 2048, 32
    per, step = C // G, 25000
    x = torch.empty((N, S, C), device="cuda", dtype=BF16)
    dy = torch.empty_like(x)
    gen = torch.Generator(device="cuda").manual_seed(71)
    for n in range(N):
        for r in range(0, S, 100000):
            xp, dp = x[n, r:r + 100000], dy[n, r:r + 100000]
            xp.copy_(torch.randn(xp.shape, generator=gen, device="cuda", dtype=BF16))
            dp.copy_(torch.randn(dp.shape, generator=gen, device="cuda", dtype=BF16))
            dp.add_(xp, alpha=0.5 + n).add_(1.0 + n)
    w = torch.rand((C,), generator=gen, device="cuda") + 0.5
    _, mean, rstd = vdf.gn_forward(x, G, w, None, EPS, out=torch.empty_like(x))
    gx, dw, db = vdf.gn_backward(x, dy, mean, rstd, G, w)
    torch.cuda.synchronize()
    say("[gn] 2^32 gradients done")

    def parts(n, r, count):
        """xhat and dy of some rows, in 64 bits, [rows, C]."""
        m, s = (t[n].double().repeat_interleave(per)[None] for t in (mean, rstd))
        return (x[n, r:r + count].double() - m) * s, dy[n, r:r + count].double()

    sums = torch.zeros((4, N, C), device="cuda", dtype=torch.float64)   # dz, dz xhat; magnitudes
    for n in range(N):
        for r in range(0, S, step):
            h, d = parts(n, r, step)
            for k, t in enumerate((d, d * h)):
                sums[k, n] += t.sum(0)
                sums[k + 2, n] += t.abs().sum(0)
    check("grad_bias", db, sums[0].sum(0).cpu(), 100 * U * sums[2].sum(0).cpu())
    check("grad_weight", dw, sums[1].sum(0).cpu(), 100 * U * sums[3].sum(0).cpu())
    means = (sums * w.double()).view(4, N, G, per).sum(3) / (S * per)
    edge = 2 ** 32 // C - S
    for n, r in ((0, 0), (0, S - 60), (1, 0), (1, edge - 30), (1, S - 60)):
        h, d = parts(n, r, 60)
        m1, m2, a1, a2 = (t.repeat_interleave(per)[None] for t in means[:, n])
        s = rstd[n].double().repeat_interleave(per)[None]
        want = s * (w.double() * d - m1 - h * m2)
        tol = s * U * (8 * (w.double() * d).abs() + 100 * (a1 + h.abs() * a2))
        check(f"grad_x of image {n} from row {r}", gx[n, r:r + 60], want.cpu(),
              rounded(tol, want, BF16).cpu())


@pytest.mark.parametrize("shape, dtype", [((2, 40003, 96, 8), F32), ((1, 30003, 192, 16), BF16),
                                          ((1, 9001, 48, 3), F16), ((1, 605, 5200, 2), F32)])
def test_mean_far_from_the_first_value_by_chunks(shape, dtype):
    """The same by chunks and by units of a wide group, where every chunk's mean is the same
    number far from the first value, so that roundings of it would not average out."""
    N, S, C, G = shape
    x = (torch.arange(C) * 7 % 8).float().expand(N, S, C).clone()
    x[:, 0, ::C // G] = 1000.0
    x = x.to(dtype).cuda()
    _, mean, rstd = vdf.gn_forward(x, G, None, None, EPS)
    torch.cuda.synchronize()
    ref = Norm(x, G, None, None, EPS, "none")
    share = 18000.0 * 16 / (S * C // G)
    check("mean", mean, ref.mean, U * (ref.mean.abs() + share))
    check("rstd", rstd, ref.rstd, ref.stat_tols()[1])
