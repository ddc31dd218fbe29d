"""The rotation, the head norm and the attention among the operators they stand between: a training
step from projections to a group norm, a serving pass of 8-bit projections with a cache of states
that grows by a token a step, eagerly and captured into graphs."""
import math

import pytest
import torch
import torch.nn.functional as F

import view_deformable_feature_amd as vdf
from attention_reference import BF16, Attention, check, norm_rotate, rounded
from gpu_helpers import say
from norm_int8_reference import codes, product

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = 2.0 ** -24


# ---- training ------------------------------------------------------------------------------

def _turn(x, freqs, pos, layout):
    a = pos.double()[..., None, None] * freqs
    R = 2 * freqs.shape[0]
    if layout == "half":
        p, q = x[..., :R // 2], x[..., R // 2:R]
        r = torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], -1)
    else:
        p, q = x[..., :R:2], x[..., 1:R:2]
        r = torch.stack([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], -1).flatten(-2)
    return torch.cat([r, x[..., R:]], -1)


def _plain_step(x, s, wq, wkv, qw, kw, gw, gb, freqs, pos, lens, mask, H, Hk, layout):
    """The step in 64 bits on the CPU, with automatic gradients."""
    B, Nq, _ = x.shape
    Nk, D = s.shape[1], qw.shape[0]
    q = (x @ wq.T).view(B, Nq, H, D)
    k, v = (s @ wkv.T).view(B, Nk, 2, Hk, D).unbind(2)

    def norm(t, w):
        return t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * w

    q = _turn(norm(q, qw), freqs, torch.arange(Nq), layout)
    k = _turn(norm(k, kw), freqs, pos, layout)
    k, v = (t.repeat_interleave(H // Hk, 2).transpose(1, 2) for t in (k, v))
    seen = mask & (torch.arange(Nk) < lens[:, None])
    score = (q.transpose(1, 2) @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(
        ~seen[:, None, None], -math.inf)
    y = (score.softmax(-1) @ v).transpose(1, 2).reshape(B, Nq, H * D)
    return F.silu(F.group_norm(y.transpose(1, 2), 4, gw, gb, 1e-5)).transpose(1, 2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("H, Hk, D", [(6, 2, 16), (4, 4, 64)])
def test_training_step(layout, H, Hk, D):
    """Gradients of all weights and inputs of projections, head norm with rotation, attention with
    lengths and a mask, and the group norm, in binary32.  The longest sum of a step has 256 terms
    (a projection), (256 + 4) 2^-24 of its terms' magnitudes at most, 1.6e-5; of eight steps, there
    and back, each passes on what came before about as it is; 8 times that is 1.3e-4 of the
    largest."""
    gen = torch.Generator().manual_seed(4201)
    B, Nq, Nk, C = 2, 37, 83, 96

    def leaf(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen) * scale + shift).cuda().requires_grad_(True)

    x, s = leaf(B, Nq, C), leaf(B, Nk, C)
    wq, wkv = leaf(H * D, C, scale=C ** -0.5), leaf(2 * Hk * D, C, scale=C ** -0.5)
    qw, kw = leaf(D, scale=0.2, shift=1.0), leaf(D, scale=0.2, shift=1.0)
    gw, gb = leaf(H * D, scale=0.2, shift=1.0), leaf(H * D, scale=0.3)
    freqs, _ = vdf.rope_frequencies(D // 2)
    pos = (torch.rand((B, Nk), generator=gen) * 60).cuda()
    lens = torch.tensor([Nk, 41], dtype=torch.int32).cuda()
    mask = (torch.rand((B, Nk), generator=gen) < 0.8).cuda()
    go = torch.randn((B, Nq, H * D), generator=gen).cuda()

    q = F.linear(x.reshape(-1, C), wq).view(B, Nq, H, D)
    k, v = F.linear(s.reshape(-1, C), wkv).view(B, Nk, 2, Hk, D).unbind(2)
    q, k = vdf.norm_rotary(q, k, qw, kw, freqs, None, pos, EPS, layout)
    y = vdf.cross_attention(q, k, v, lens, mask)
    out = vdf.group_norm_act(y.reshape(B, Nq, H * D), 4, gw, gb, activation="silu")
    leaves = (x, s, wq, wkv, qw, kw, gw, gb)
    grads = torch.autograd.grad((out * go).sum(), leaves)
    torch.cuda.synchronize()

    plain = [t.detach().cpu().double().requires_grad_(True) for t in leaves]
    ref = _plain_step(*plain, freqs.cpu(), pos.cpu(), lens.cpu(), mask.cpu(), H, Hk, layout)
    want = torch.autograd.grad((ref * go.cpu().double()).sum(), plain)
    tol = 1.3e-4
    check("out", out.detach(), ref.detach(), torch.full_like(ref, tol * float(ref.detach().abs().max())))
    for name, a, b in zip("x s wq wkv qw kw gw gb".split(), grads, want):
        check(name, a, b, torch.full_like(b, tol * float(b.abs().max())))


def test_training_step_captured():
    """Forward and gradients in a graph, replayed with eager steps of other leaves between."""
    gen = torch.Generator().manual_seed(4202)
    B, Nq, Nk, H, Hk, D = 2, 45, 130, 8, 4, 64
    q0, go = (torch.randn((B, Nq, H, D), generator=gen).to(BF16).cuda() for _ in range(2))
    k0, v0 = (torch.randn((B, Nk, Hk, D), generator=gen).to(BF16).cuda() for _ in range(2))
    w0 = (torch.rand(D, generator=gen) + 0.5).cuda()
    freqs, _ = vdf.rope_frequencies(D)
    lens = torch.tensor([Nk, 70], dtype=torch.int32).cuda()

    def step(leaves):
        q, k, v, w = leaves
        a, b = vdf.norm_rotary(q, k, w, w, freqs)
        y = vdf.cross_attention(a, b, v, lens)
        return (y, *torch.autograd.grad(y, leaves, go))

    def fresh():
        return [t.detach().clone().requires_grad_(True) for t in (q0, k0, v0, w0)]

    held = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for n in range(4):
        q0.mul_(1.2)
        lens.copy_(torch.tensor([Nk - 30 * n, 40 * n], dtype=torch.int32))
        with torch.no_grad():
            held[0].copy_(q0)
        for t in got:
            t.detach().fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want = step(fresh())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {n}"


# ---- serving -------------------------------------------------------------------------------

class Layer:
    """8-bit projections around attention to a cache of rotated keys and of values."""

    def __init__(self, C, H, Hk, D, B, room, seed):
        gen = torch.Generator().manual_seed(seed)

        def weights(n, c):
            return vdf.i8_quantize_rows((torch.randn((n, c), generator=gen) * c ** -0.5).cuda())

        self.C, self.H, self.Hk, self.D, self.B = C, H, Hk, D, B
        self.qkv, self.back = weights((H + 2 * Hk) * D, C), weights(C, H * D)
        self.qw, self.kw = ((torch.rand(D, generator=gen) + 0.5).cuda() for _ in range(2))
        self.freqs, self.magnitude = vdf.rope_frequencies(D, scaling="blend", factor=4.0, trained=64)
        self.keys, self.values = (torch.full((B, room, Hk, D), math.nan, dtype=BF16, device="cuda")
                                  for _ in range(2))

    def project(self, x):
        B, N, _ = x.shape
        heads = vdf.i8_linear(x, *self.qkv, out_dtype=BF16).view(B, N, self.H + 2 * self.Hk, self.D)
        return heads.split([self.H, self.Hk, self.Hk], 2)

    def attend(self, q, lens):
        y, _ = vdf.attn_forward(q, self.keys, self.values, lens)
        return vdf.i8_linear(y.view(*y.shape[:2], -1), *self.back, out_dtype=BF16)

    def prompt(self, x, lens):
        """The first N states of the cache; positions 0, 1, 2, ..."""
        N = x.shape[1]
        q, k, v = self.project(x)
        self.values[:, :N].copy_(v)
        vdf.rope_norm_forward(q, k, self.qw, self.kw, self.freqs, None, None, EPS, "half",
                              self.magnitude, q_out=q, k_out=self.keys[:, :N])
        return q, self.attend(q, lens)

    def token(self, x, lens):
        """One token for each entry, at its own length, which counts it already."""
        q, k, v = self.project(x)
        at = (lens - 1).view(self.B, 1)
        vdf.rope_norm_forward(q, k, self.qw, self.kw, self.freqs, at, at, EPS, "half",
                              self.magnitude, q_out=q, k_out=k)
        place = at.long().view(self.B, 1, 1, 1).expand(-1, 1, self.Hk, self.D)
        self.keys.scatter_(1, place, k)
        self.values.scatter_(1, place, v)
        return q, self.attend(q, lens)


@pytest.mark.parametrize("C, H, Hk, D, N", [(64, 4, 2, 32, 21), (256, 8, 8, 64, 150), (192, 6, 1, 128, 33)])
def test_serving_pass(C, H, Hk, D, N):
    """A ragged prompt, then single tokens; each step against its definition, from what the step before it gave.
    What the cache does not hold yet are NaN."""
    say(f"[serving] {C} {H} {Hk} {D} {N}")
    B, room = 3, N + 6
    gen = torch.Generator().manual_seed(4203)
    layer = Layer(C, H, Hk, D, B, room, 4204)
    lens = torch.tensor([N, 1, N // 2], dtype=torch.int32).cuda()
    x = torch.randn((B, N, C), generator=gen).to(BF16).cuda()

    def checked(x, step, pos):
        before = layer.project(x)
        q, out = step(x, lens)
        torch.cuda.synchronize()
        n = x.shape[1]
        rows = x.reshape(-1, C)
        ref, tol = product(*codes(rows), *layer.qkv, None, "none")
        got = torch.cat([t.reshape(B * n, -1) for t in before], 1)
        check("projection", got, ref, rounded(tol, ref, BF16))
        check("q", q, *norm_rotate(before[0], layer.qw, layer.freqs, pos, "half", EPS, layer.magnitude))
        want, tol = norm_rotate(before[1], layer.kw, layer.freqs, pos, "half", EPS, layer.magnitude)
        for b in range(B):
            at = pos[b].long().cpu()
            check(f"keys {b}", layer.keys[b, at], want[b], tol[b])
            assert torch.equal(layer.values[b, at.cuda()], before[2][b])
        y, lse = vdf.attn_forward(q, layer.keys, layer.values, lens)
        torch.cuda.synchronize()
        Attention(q, layer.keys, layer.values, lens).check_forward(y, lse)
        ref, tol = product(*codes(y.reshape(B * n, -1)), *layer.back, None, "none")
        check("out", out.reshape(B * n, -1), ref, rounded(tol, ref, BF16))

    checked(x, layer.prompt, torch.arange(N).repeat(B, 1))
    for _ in range(3):
        lens.add_(1)
        x = torch.randn((B, 1, C), generator=gen).to(BF16).cuda()
        checked(x, layer.token, (lens - 1).view(B, 1).cpu())


def test_tokens_captured_on_two_streams():
    """Two caches' steps in graphs of their own, replayed at once on two streams, token after token,
    with the same steps eagerly on copies of the caches between the replays."""
    B, C, H, Hk, D, room = 4, 128, 8, 2, 64, 3000
    gen = torch.Generator().manual_seed(4205)
    layers, copies, graphs, held = [], [], [], []
    for n in range(2):
        pair = [Layer(C, H, Hk, D, B, room, 4206 + n) for _ in range(2)]
        for layer in pair:
            layer.keys.copy_(torch.randn((B, room, Hk, D), generator=gen.manual_seed(n)).to(BF16))
            layer.values.copy_(torch.randn((B, room, Hk, D), generator=gen.manual_seed(9 + n)).to(BF16))
        layers.append(pair[0]), copies.append(pair[1])
    lens = torch.tensor([1, 2990, 700, 2048], dtype=torch.int32).cuda()
    for layer in layers:
        x = torch.randn((B, 1, C), generator=gen).to(BF16).cuda()
        keys, values = layer.keys.clone(), layer.values.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.token(x, lens)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = layer.token(x, lens)
        layer.keys.copy_(keys), layer.values.copy_(values)
        graphs.append(graph), held.append((x, got))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for n in range(4):
        lens.add_(1)
        for x, got in held:
            x.copy_(torch.randn((B, 1, C), generator=gen).to(BF16))
            for t in got:
                t.fill_(math.nan)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (x, got), layer, copy in zip(held, layers, copies):
            want = copy.token(x, lens)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {n}"
            assert torch.equal(layer.keys, copy.keys) and torch.equal(layer.values, copy.values)


def test_on_a_stream_that_is_not_the_current_one_of_its_tensors():
    """Work queued on a side stream behind what fills its inputs there, results read there."""
    gen = torch.Generator().manual_seed(4207)
    host = [torch.randn((2, n, h, 64), generator=gen).to(BF16).pin_memory()
            for n, h in ((500, 8), (500, 2), (500, 2))]
    freqs, _ = vdf.rope_frequencies(64)

    def work():
        q, k, v = (t.to("cuda", non_blocking=True) for t in host)
        q, k = vdf.rope_norm_forward(q, k, None, None, freqs)
        out, lse = vdf.attn_forward(q, k, v)
        return (out, lse, *vdf.attn_backward(q, k, v, out, lse, out))

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_rotation_of_what_turns_back():
    """Queries rotated by far positions and back are themselves.  With p the sum of a pair's two
    magnitudes a turn is off by 8 u times at most 2 p; of two such errors the turn back makes no
    more than sqrt(2) times one, 23 u p, and adds its own of a pair whose sum is at most sqrt(2) p,
    23 u p."""
    x = torch.randn((2, 40, 3, 96), generator=torch.Generator().manual_seed(4208)).cuda()
    freqs, _ = vdf.rope_frequencies(96)
    pos = torch.arange(40).cuda() + 900000
    y = vdf.rotary(x, freqs, pos, "interleaved")
    back = vdf.rope_forward(y, freqs, pos, "interleaved", inverse=True)
    torch.cuda.synchronize()
    ref = x.double().cpu()
    p = (ref[..., ::2].abs() + ref[..., 1::2].abs()).repeat_interleave(2, -1)
    check("back", back, ref, 46 * U * p)
