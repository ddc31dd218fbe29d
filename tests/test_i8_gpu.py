"""8-bit codes and their products on the GPU against the definition in 64 bits
(norm_int8_reference.py has the bounds): sizes around every tile and vector, one row and
many, extreme codes at the longest sum, rows of zeros, of tiny numbers and with NaNs, types
and activations, views off alignment, streams and graphs, and the normalised form."""
import numpy as np
import pytest
import torch

import view_deformable_feature_amd as vdf
from gpu_helpers import say
from norm_int8_reference import U, Norm, act, check, codes, gelu_tols, product, rounded

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _layer(N, K, seed, bias=True):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8)
    scale = torch.rand((N,), generator=gen) * 0.01 + 1e-3
    b = torch.randn((N,), generator=gen) if bias else None
    return tuple(None if t is None else t.cuda() for t in (w, scale, b))


def _rows(M, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=gen) * (torch.rand((M, 1), generator=gen) * 3 + 0.01)
    return x.to(dtype).cuda()


def _codes(M, K, seed):
    gen = torch.Generator().manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), generator=gen, dtype=torch.int8)
    return a.cuda(), (torch.rand((M,), generator=gen) * 0.05 + 1e-3).cuda()


SIZES = [(1, 1, 1), (1, 64, 16), (2, 3, 5), (1, 4096, 33), (3, 1000, 777), (5, 16, 64), (15, 65, 17),
         (16, 128, 108), (17, 127, 63), (31, 256, 128), (33, 80, 130), (64, 64, 64), (65, 48, 256),
         (100, 520, 100), (127, 129, 127), (128, 128, 128), (129, 1024, 129), (200, 2000, 300),
         (255, 192, 257), (256, 512, 256), (300, 31, 40), (513, 272, 200), (900, 256, 2496),
         (1237, 1000, 77), (4100, 128, 108), (777, 4096, 513), (20011, 16, 3), (6, 512, 5000)]


@pytest.mark.parametrize("M, K, N", SIZES)
def test_matmul_sizes(M, K, N):
    say(f"[i8] matmul {M} {K} {N}")
    a, s = _codes(M, K, M + K)
    w, ws, b = _layer(N, K, N + K, bias=N % 2 == 0)
    out = vdf.i8_matmul(a, s, w, ws, b)
    torch.cuda.synchronize()
    ref, tol = product(a, s, w, ws, b, "none")
    assert out.dtype == F32
    check("out", out, ref, tol)


@pytest.mark.parametrize("M, K, N", SIZES)
def test_linear_sizes(M, K, N):
    """The same numbers as quantising and multiplying one after the other."""
    say(f"[i8] linear {M} {K} {N}")
    dtype = (F32, BF16, F16)[(M + K + N) % 3]
    x = _rows(M, K, dtype, M * 3 + K)
    w, ws, b = _layer(N, K, N * 5 + K, bias=N % 2 == 1)
    out = vdf.i8_linear(x, w, ws, b)
    q, s = vdf.i8_quantize_rows(x)
    both = vdf.i8_matmul(q, s, w, ws, b)
    torch.cuda.synchronize()
    qr, sr = codes(x)
    assert torch.equal(q.cpu(), qr) and torch.equal(s.cpu(), sr)
    ref, tol = product(qr, sr, w, ws, b, "none")
    check("out", out, ref, tol)
    assert torch.equal(out, both)


@pytest.mark.parametrize("M, K, N", [(3950, 384, 3990), (3950, 128, 3985), (3841, 256 + 128, 4100),
                                     (25700, 640, 510), (3950, 300, 3990), (3950, 272, 4001)])
@pytest.mark.parametrize("out_dtype", [F32, BF16], ids=["f32", "bf16"])
def test_large_products(M, K, N, out_dtype):
    """Enough 256 x 256 tiles to fill the card, with ragged edges, and the columns that keep
    such a product on smaller tiles."""
    say(f"[i8] large {M} {K} {N} {out_dtype}")
    a, s = _codes(M, K, 201)
    w, ws, b = _layer(N, K, 202)
    out = vdf.i8_matmul(a, s, w, ws, b, activation="relu", out_dtype=out_dtype)
    torch.cuda.synchronize()
    ref, tol = product(a, s, w, ws, b, "relu")
    check("out", out, ref, rounded(tol, ref, out_dtype))


@pytest.mark.parametrize("act_name", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("out_dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [2, 150, 700])
def test_activations_and_types(act_name, out_dtype, M):
    x = _rows(M, 200, BF16, 71)
    w, ws, b = _layer(136, 200, 72)
    ws = ws * 0.05
    out = vdf.i8_linear(x, w, ws, b, activation=act_name, out_dtype=out_dtype)
    torch.cuda.synchronize()
    ref, tol = product(*codes(x), w, ws, b, act_name)
    assert out.dtype == out_dtype
    check("out", out, ref, rounded(tol, ref, out_dtype))


@pytest.mark.parametrize("M", [1, 3, 70, 300])
def test_extreme_codes_at_the_longest_sum(M):
    """131071 products of -128 by -128 stay below 2^31."""
    K, N = 131071, 20
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    out = vdf.i8_matmul(a, one[:M], w, one[:N])
    torch.cuda.synchronize()
    want = torch.tensor([131071.0 * 16384, -131071.0 * 16256]).repeat(N // 2).float()
    assert torch.equal(out.cpu(), want.expand(M, N))
    with pytest.raises(vdf._lib.DAError):
        vdf.i8_matmul(torch.zeros((1, K + 1), dtype=torch.int8, device="cuda"), one[:1],
                      torch.zeros((1, K + 1), dtype=torch.int8, device="cuda"), one[:1])


@pytest.mark.parametrize("K", [1, 7, 8, 64, 100, 128, 500, 512, 513, 1024, 2048, 4096, 5000, 20000])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_quantize(K, dtype):
    x = _rows(37, K, dtype, 80 + K)
    x[3] = 0
    x[5] = x[5].abs() * 0 + (1e-4 if dtype == F16 else 1e-20)
    x[7, K // 2] = 0
    if dtype != F16:
        x[9] = 2.0 ** -101                       # below the smallest that has codes
        x[10] = 2.0 ** -100
        x[11, K - 1] = 3e38
    x[13, :] = torch.arange(K, device="cuda").remainder(255).sub(127).to(dtype)   # halves to even
    x[14, :] = torch.arange(K, device="cuda").remainder(255).sub(127).to(dtype) * 0.5
    x[15, K - 1] = float("nan")
    x[16, 0] = float("inf")
    x[17, K // 2] = -float("inf")
    q, s = vdf.i8_quantize_rows(x)
    torch.cuda.synchronize()
    qr, sr = codes(x)
    assert torch.equal(q.cpu(), qr)
    assert torch.equal(s.cpu().isnan(), sr.isnan())
    assert torch.equal(s.cpu().nan_to_num(), sr.nan_to_num())
    assert int(s.isnan().sum()) == 3


@pytest.mark.parametrize("M, K, N", [(1, 256, 40), (30, 256, 40), (500, 256, 200), (40, 1500, 64),
                                     (300, 1500, 130)])
def test_bad_rows_stay_in_their_row(M, K, N):
    x = _rows(M, K, F32, 90)
    x[M // 2, K // 3] = float("nan")
    if M > 1:
        x[0, K - 1] = float("inf")
        x[M - 1] = 0
    w, ws, b = _layer(N, K, 91)
    out = vdf.i8_linear(x, w, ws, b)
    torch.cuda.synchronize()
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[M // 2] = True
    if M > 1:
        bad[0] = True
        assert torch.equal(out[M - 1], b)
    assert out[bad].isnan().all() and not out[~bad].isnan().any()


@pytest.mark.parametrize("M, K, N", [(3, 256, 64), (200, 256, 136), (700, 128, 108)])
def test_views_off_alignment(M, K, N):
    def shifted(t):
        v = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:].view(t.shape)
        return v.copy_(t)

    x = _rows(M, K, BF16, 95)
    w, ws, b = _layer(N, K, 96)
    want = vdf.i8_linear(x, w, ws, b)
    q, s = vdf.i8_quantize_rows(x)
    for xi, wi in ((shifted(x), w), (x, shifted(w)), (shifted(x), shifted(w))):
        got = vdf.i8_linear(xi, wi, shifted(ws), shifted(b), out=shifted(want).fill_(float("nan")))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    got = vdf.i8_matmul(shifted(q), shifted(s), w, ws, b)
    half = vdf.i8_matmul(q, s, w, ws, b, out=shifted(want.half()))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(half, want.half())


def test_leading_dimensions_and_empty():
    x = _rows(24, 64, F32, 97).view(2, 3, 4, 64)
    w, ws, b = _layer(10, 64, 98)
    out = vdf.i8_linear(x, w, ws, b)
    one = vdf.i8_linear(x[0, 0, 0], w, ws, b)
    none = vdf.i8_linear(x[:0], w, ws, b)
    q, s = vdf.i8_quantize_rows(x[:0])
    nothing = vdf.i8_matmul(q, s, w, ws, b)
    torch.cuda.synchronize()
    assert out.shape == (2, 3, 4, 10) and one.shape == (10,) and torch.equal(one, out[0, 0, 0])
    assert none.shape == (0, 3, 4, 10) and nothing.shape == none.shape


def _norm_linear_ref(x, G, nw, nb, eps, act_name, w, ws, b):
    """(out, bound): where a normalised value lies within its bound of a half, its code may be
    either of two; elsewhere codes agree, and a row's scale is off by its largest value's
    bound."""
    ref = Norm(x, G, nw, nb, eps, act_name)
    N, S, C = x.shape
    y, ytol = ref.y.reshape(N * S, C), (2 * ref.ztol).reshape(N * S, C)
    big = y.abs().amax(1, keepdim=True)
    top = (ytol + 0 * y).amax(1, keepdim=True)           # bound of big
    some = big > 4 * top                                  # a row of a rectifier may be all zeros
    safe = torch.where(some, big, torch.ones_like(big))
    t = torch.where(some, y * (127 / safe), torch.zeros_like(y))
    ttol = torch.where(some, 127 / safe * (ytol + y.abs() * (top / safe + 4 * U)), torch.zeros_like(y))
    q = torch.round(t)
    may = ((t - torch.floor(t) - 0.5).abs() <= ttol).double()
    wd = w.cpu().double() * ws.cpu().double()[:, None]
    scale = torch.where(some, big / 127, torch.zeros_like(big))
    out = (q @ wd.t()) * scale
    mag = (q.abs() @ wd.abs().t()) * scale
    tol = (may @ wd.abs().t()) * scale + mag * (torch.where(some, top / safe, torch.zeros_like(top)) + 8 * U)
    # rows left out above: all their values are within 4 bounds of zero
    tol = tol + torch.where(some, torch.zeros_like(big), 6 * top) @ wd.abs().sum(1)[None, :]
    if b is not None:
        out = out + b.cpu().double()
        tol = tol + 8 * U * b.cpu().double().abs()
    return out, tol + 8 * U * out.abs() + 2.0 ** -140


NORM_SIZES = [(1, 1, 64, 2, 9), (2, 33, 64, 8, 27), (3, 50, 128, 32, 108), (1, 196, 512, 32, 432),
              (2, 784, 256, 32, 216), (2, 45, 21, 3, 10), (1, 300, 96, 16, 64), (5, 17, 512, 4, 33),
              (2, 20, 640, 5, 40), (1, 9, 1024, 8, 70), (1, 5, 4096, 2, 12), (40, 3, 32, 4, 130),
              (2, 700, 128, 4, 1000), (1, 20003, 16, 2, 5)]


@pytest.mark.parametrize("N, S, C, G, D", NORM_SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_norm_linear(N, S, C, G, D, dtype):
    say(f"[i8] norm linear {N} {S} {C} {G} {D} {dtype}")
    gen = torch.Generator().manual_seed(N + S + C)
    x = (torch.randn((N, S, C), generator=gen) * 1.3 + 0.4).to(dtype).cuda()
    nw = (torch.rand((C,), generator=gen) + 0.5).cuda()
    nb = (torch.randn((C,), generator=gen) * 0.3).cuda()
    w, ws, b = _layer(D, C, D + C, bias=D % 2 == 0)
    out = vdf.i8_norm_linear(x, G, nw, nb, w, ws, b, activation="silu")
    torch.cuda.synchronize()
    ref, tol = _norm_linear_ref(x, G, nw, nb, 1e-5, "silu", w, ws, b)
    check("out", out, ref.view(N, S, D), tol.view(N, S, D))


@pytest.mark.parametrize("act_name", ["none", "relu", "gelu"])
@pytest.mark.parametrize("params", [True, False], ids=["affine", "plain"])
def test_norm_linear_activations(act_name, params):
    gen = torch.Generator().manual_seed(101)
    x = torch.randn((2, 3, 21, 64), generator=gen).cuda()
    nw = (torch.rand((64,), generator=gen) + 0.5).cuda() if params else None
    nb = torch.randn((64,), generator=gen).cuda() if params else None
    w, ws, b = _layer(48, 64, 102)
    out = vdf.i8_norm_linear(x, 8, nw, nb, w, ws, b, activation=act_name, out_dtype=BF16)
    torch.cuda.synchronize()
    ref, tol = _norm_linear_ref(x.view(2, 63, 64), 8, nw, nb, 1e-5, act_name, w, ws, b)
    assert out.shape == (2, 3, 21, 48) and out.dtype == BF16
    check("out", out, ref, rounded(tol, ref, BF16))


def test_norm_linear_rows_without_a_positive_value():
    """Rows that the rectifier empties: the projection's bias."""
    x = torch.randn((1, 40, 32), device="cuda")
    x[0, ::2] = -10
    nb = torch.full((32,), -1.0, device="cuda")
    w, ws, b = _layer(20, 32, 103)
    out = vdf.i8_norm_linear(x, 1, None, nb, w, ws, b, activation="relu")
    torch.cuda.synchronize()
    assert torch.equal(out[0, ::2], b.expand(20, 20))


def test_norm_linear_bad_values_stay_in_their_image():
    x = torch.randn((3, 70, 64), device="cuda")
    x[1, 20, 40] = float("nan")
    w, ws, b = _layer(24, 64, 104)
    out = vdf.i8_norm_linear(x, 4, None, None, w, ws, b)
    torch.cuda.synchronize()
    assert out[1].isnan().all() and not out[0].isnan().any() and not out[2].isnan().any()


def test_norm_linear_views_off_alignment():
    buf = torch.randn(2 * 90 * 64 + 1, device="cuda")
    x = buf[1:].view(2, 90, 64)
    w, ws, b = _layer(24, 64, 105)
    wv = torch.empty(24 * 64 + 1, device="cuda", dtype=torch.int8)[1:].view(24, 64).copy_(w)
    got = vdf.i8_norm_linear(x, 4, None, None, wv, ws, b, activation="silu")
    torch.cuda.synchronize()
    ref, tol = _norm_linear_ref(x, 4, None, None, 1e-5, "silu", w, ws, b)
    check("out", got, ref, tol)
    assert vdf.i8_norm_linear(x[:0], 4, None, None, w, ws, b).shape == (0, 90, 24)


def test_repeatable_and_another_stream():
    x = _rows(3000, 640, BF16, 110)
    w, ws, b = _layer(300, 640, 111)
    want = vdf.i8_linear(x, w, ws, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p = [vdf.i8_linear(x, w, ws, b) for _ in range(3)]
    q = [vdf.i8_linear(x, w, ws, b) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in p + q)


@pytest.mark.parametrize("M, K, N", [(1, 4096, 512), (8, 2048, 1000), (700, 256, 108), (300, 1500, 64)])
def test_graph_replays_match_eager(M, K, N):
    x = _rows(M, K, F16, 112)
    w, ws, b = _layer(N, K, 113)
    nx = _rows(M, 64, F32, 114).view(1, M, 64)
    pw, ps, pb = _layer(40, 64, 115)

    def step():
        q, s = vdf.i8_quantize_rows(x)
        return (vdf.i8_linear(x, w, ws, b), vdf.i8_matmul(q, s, w, ws, b, activation="silu"),
                vdf.i8_norm_linear(nx, 8, None, None, pw, ps, pb, activation="silu"))

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
        x.copy_(first).mul_(1 + 0.5 * k)
        nx.mul_(0.75)
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, t) for p, t in zip(got, want)), f"replay {k}"


def test_reference_by_hand():
    """Two rows and two weights worked out by hand."""
    x = torch.tensor([[1.27, -0.635, 0.0], [0.0, 254.0, 127.0]], device="cuda")
    q, s = vdf.i8_quantize_rows(x)
    w = torch.tensor([[1, 2, 3], [-4, 0, 5]], dtype=torch.int8, device="cuda")
    ws = torch.tensor([0.5, 2.0], device="cuda")
    out = vdf.i8_matmul(q, torch.tensor([0.01, 2.0], device="cuda"), w, ws)
    torch.cuda.synchronize()
    assert q.cpu().tolist()[1] == [0, 127, 64]              # 63.5 goes to the even 64
    assert q.cpu().tolist()[0][0] == 127 and q.cpu().tolist()[0][2] == 0
    assert float(s[1]) == 2.0
    k = q.cpu().tolist()[0][1]
    assert k in (-63, -64)
    want = [[(127 + 2 * k) * 0.01 * 0.5, -508 * 0.01 * 2.0], [446 * 2.0 * 0.5, 320 * 2.0 * 2.0]]
    assert np.allclose(out.cpu().numpy(), np.array(want), rtol=1e-6)
    assert act(torch.tensor(-1.0), "relu") == 0


def test_more_values_than_32_bits_count():
    """17 million rows of 256 numbers: places past 2^32 of x, and of the result."""
    M, K, N = 17_000_003, 256, 260
    x = torch.empty((M, K), device="cuda", dtype=BF16)
    gen = torch.Generator(device="cuda").manual_seed(120)
    for r in range(0, M, 1 << 20):
        part = x[r:r + (1 << 20)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=BF16))
    w, ws, b = _layer(N, K, 121)
    out = vdf.i8_linear(x, w, ws, b, out_dtype=BF16)
    last = vdf.i8_linear(x[-1000:].contiguous(), w, ws, b, out_dtype=BF16)
    q, s = vdf.i8_quantize_rows(x)
    ql, sl = vdf.i8_quantize_rows(x[-1000:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(out[-1000:], last)
    assert torch.equal(q[-1000:], ql) and torch.equal(s[-1000:], sl)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gelu_keeps_its_digits_in_the_lower_tail(M):
    """z = k / 16 exactly, from -7.94 to 7.94, of one code times one weight: K = 1 and, of rows
    that are zero but for one column, 300."""
    for K in (1, 300):
        a = torch.zeros((M, K), dtype=torch.int8, device="cuda")
        a[:, 0] = 1
        w = torch.zeros((255, K), dtype=torch.int8, device="cuda")
        w[:, 0] = torch.arange(-127, 128, device="cuda")
        out = vdf.i8_matmul(a, torch.full((M,), 0.25, device="cuda"), w,
                            torch.full((255,), 0.25, device="cuda"), activation="gelu")
        torch.cuda.synchronize()
        z = (torch.arange(-127, 128).double() / 16).expand(M, 255)
        check("out", out, act(z, "gelu"), gelu_tols(z)[0])


@pytest.mark.parametrize("M, K, N", [(3950, 384, 3990), (300, 520, 100), (300, 384, 129),
                                     (100, 2048, 300), (20, 1000, 70), (40, 520, 33), (9, 300, 50)])
def test_codes_off_alignment(M, K, N):
    """Codes one byte into larger buffers, scales, bias and result one element: 256 x 256 tiles
    (which take only aligned codes), 64 x 64 tiles and the streaming kernel at 16, 32 and 64 rows
    a workgroup give what they give for aligned ones, bit for bit."""
    say(f"[i8] off alignment {M} {K} {N}")

    def shifted(t):
        v = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:].view(t.shape)
        return v.copy_(t)

    a, s = _codes(M, K, 130)
    w, ws, b = _layer(N, K, 131)
    want = vdf.i8_matmul(a, s, w, ws, b, activation="silu")
    x = _rows(M, K, BF16, 132)
    linear = vdf.i8_linear(x, w, ws, b)
    torch.cuda.synchronize()
    ref, tol = product(a, s, w, ws, b, "silu")
    check("aligned", want, ref, tol)
    for ai, wi in ((shifted(a), w), (a, shifted(w)), (shifted(a), shifted(w))):
        got = vdf.i8_matmul(ai, shifted(s), wi, shifted(ws), shifted(b), activation="silu",
                            out=shifted(want).fill_(float("nan")))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    got = vdf.i8_linear(shifted(x), shifted(w), shifted(ws), shifted(b))
    half = vdf.i8_matmul(shifted(a), s, w, ws, b, activation="silu", out=shifted(want.half()))
    torch.cuda.synchronize()
    assert torch.equal(got, linear) and torch.equal(half, want.half())


def test_norm_linear_with_weights_off_alignment():
    """Behind a norm: 256 x 256 tiles' worth of rows with weights at an odd address."""
    x = torch.randn((2, 16500, 384), device="cuda")
    w, ws, b = _layer(256, 384, 133)
    wv = torch.empty(256 * 384 + 1, device="cuda", dtype=torch.int8)[1:].view(256, 384).copy_(w)
    want = vdf.i8_norm_linear(x, 8, None, None, w, ws, b, activation="silu")
    got = vdf.i8_norm_linear(x, 8, None, None, wv, ws, b, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(got, want)
