"""What is measured of the normalisation and the 8-bit product operators, and their plain forms.

Four operators on channels-last maps, [images, rows, C] with one row per pixel (or
[tokens, C] where nothing is normalised):

* ``gn_forward``: group norm over (rows, C / groups), the affine map per channel and an
  activation;
* ``gn_backward``: its gradients;
* ``i8_matmul``: the product of 8-bit codes with a scale per row and per output channel;
* ``i8_linear``: the same for rows in 16 or 32 bits, each quantised to 8 bits by its
  largest magnitude within the call;
* ``i8_norm_linear``: group norm, activation and ``i8_linear`` in one call, the serving
  form of a normalised map that goes into a 1x1 projection.

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits,
with ``own`` true through this package.  ``exact`` gives the same in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-5


def listed():
    return [
        # the coarsest level of a six-camera pyramid: a call of a few microseconds
        dict(name="norm_level_8x22", op="norm", N=6, S=8 * 22, C=256, G=8, act="relu", dtype="f32"),
        # a training batch of the 56x56x128 stage that deformable convolutions run in
        dict(name="norm_56x56", op="norm", N=64, S=56 * 56, C=128, G=32, act="silu", dtype="bf16"),
        # the finest level of the six-camera pyramid, whole in 32 bits
        dict(name="norm_level_64x176", op="norm", N=6, S=64 * 176, C=256, G=32, act="relu",
             dtype="f32"),
        # the backward pass of a training batch of the 28x28x256 stage
        dict(name="norm_grad_28x28", op="norm_grad", N=64, S=28 * 28, C=256, G=32, act="silu",
             dtype="bf16"),
        # a ragged map with three groups of 32 channels
        dict(name="norm_grad_37x45", op="norm_grad", N=3, S=37 * 45, C=96, G=3, act="gelu",
             dtype="f16"),
        # 900 anchors of 256 channels to 13 points x 6 cameras x 4 scales x 8 groups of weights
        dict(name="matmul_900_anchors", op="matmul", M=900, K=256, N=13 * 6 * 4 * 8, bias=True,
             act="none", out="f32"),
        # a large product, bound by the matrix cores
        dict(name="matmul_8192", op="matmul", M=8192, K=4096, N=4096, bias=False, act="none",
             out="bf16"),
        # one token: the weights are read once and little is computed
        dict(name="linear_one_token", op="linear", M=1, K=4096, N=4096, bias=True, act="none",
             dtype="bf16", out="bf16"),
        # offsets and scalars of a 56x56 deformable convolution, 4 groups of 3 x 9 numbers
        dict(name="linear_offsets_56x56", op="linear", M=64 * 56 * 56, K=128, N=4 * 27, bias=True,
             act="none", dtype="bf16", out="f32"),
        # odd sizes everywhere
        dict(name="linear_odd", op="linear", M=1237, K=1000, N=777, bias=True, act="gelu",
             dtype="f16", out="f16"),
        # a normalised 28x28x256 batch into 8 groups of 27 offsets and scalars
        dict(name="norm_linear_28x28", op="norm_linear", N=64, S=28 * 28, C=256, G=32, act="silu",
             D=8 * 27, bias=True, dtype="bf16", out="bf16"),
        # one image of the 14x14x512 stage, 16 groups
        dict(name="norm_linear_14x14", op="norm_linear", N=1, S=14 * 14, C=512, G=32, act="silu",
             D=16 * 27, bias=True, dtype="f16", out="f16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def _map(rng, most, channels, least):
    """Images, rows, channels and groups: at most `most` values, and `least` to a group (of a few
    values each is its mean but for rounding, and the gradient of their normalised form is the
    small difference of large numbers)."""
    per = rng.choice([1, 2, 3, 4, 8, 8, 12, 16, 24, 32, 32, 64])
    G = _spread(rng, 1, max(1, min(32, channels // per)))
    N = _spread(rng, 1, 64)
    S = _spread(rng, 1, max(1, min(most // (N * G * per), 200 * 400)))
    return dict(N=N, S=max(S, -(-least // per)), C=G * per, G=G)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "matmul", "linear", "norm_linear"])
    dtype, out = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "bf16", "f16"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    bias = rng.random() < 0.7
    if op == "norm":
        most = (1 << 24) if dtype == "f32" else (1 << 24) + (1 << 23)
        return dict(op=op, act=act, dtype=dtype, **_map(rng, most, 512, 16))
    if op == "norm_grad":
        # relu is left out: where its argument is a rounding away from zero, its derivative is
        # either of two values, and of many million arguments some always are
        act = rng.choice(["none", "silu", "gelu"])
        return dict(op=op, act=act, dtype=dtype, **_map(rng, 1 << 23, 512, 64))
    if op == "norm_linear":
        # out in 16 bits, as serving has it: a code that rounding moves by one changes more
        # than the last bits of a 32-bit result
        dtype, out = rng.choice(["bf16", "f16"]), rng.choice(["bf16", "f16"])
        m = _map(rng, 1 << 23, 512, 16)
        D = _spread(rng, 1, max(1, min(1024, (1 << 25) // (m["N"] * m["S"]))))
        return dict(op=op, act=act, dtype=dtype, out=out, D=D, bias=bias, **m)
    K, N = _spread(rng, 1, 4096), _spread(rng, 1, 4096)
    M = _spread(rng, 1, max(1, min(1 << 18, (1 << 25) // (K + N), (1 << 36) // (K * N))))
    if op == "matmul":
        return dict(op=op, M=M, K=K, N=N, bias=bias, act=act, out=out)
    return dict(op=op, M=M, K=K, N=N, bias=bias, act=act, dtype=dtype, out=out)


def _maps(case, gen):
    """A map with a mean and a spread of its own in each channel, and the affine parameters."""
    N, S, C = case["N"], case["S"], case["C"]
    dev = "cuda"
    x = torch.randn((N, S, C), generator=gen, device=dev)
    x *= torch.rand((C,), generator=gen, device=dev) * 1.5 + 0.5
    x += torch.randn((C,), generator=gen, device=dev) * 0.5 + 0.4
    return dict(x=x.to(_TYPES[case["dtype"]]),
                weight=torch.rand((C,), generator=gen, device=dev) + 0.5,
                bias=torch.randn((C,), generator=gen, device=dev) * 0.3)


def _weights(N, K, bias, gen):
    """A layer's weights as 8-bit codes with a scale per output channel, and its bias."""
    w = torch.randn((N, K), generator=gen, device="cuda") / math.sqrt(K)
    scale = (w.abs().amax(1) / 127).clamp_min(1e-20)
    codes = (w / scale[:, None]).round().clamp(-127, 127).to(torch.int8)
    b = torch.randn((N,), generator=gen, device="cuda") * 0.1 if bias else None
    return dict(w=codes, w_scale=scale, b=b)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case=case)
    if op in ("norm", "norm_grad", "norm_linear"):
        state.update(_maps(case, gen))
        if op == "norm_linear":
            state.update(_weights(case["D"], case["C"], case["bias"], gen))
        if op == "norm_grad":
            # what the forward pass kept, and the gradient that comes back
            x = state["x"].float().view(case["N"], case["S"], case["G"], -1)
            mean = x.mean((1, 3), dtype=torch.float64)
            var = (x.double() - mean[:, None, :, None]).square().mean((1, 3))
            state["mean"] = mean.float()
            state["rstd"] = (var + _EPS).rsqrt().float()
            state["grad"] = torch.randn(state["x"].shape, generator=gen,
                                        device="cuda").to(state["x"].dtype)
        return state
    M, K, N = case["M"], case["K"], case["N"]
    state.update(_weights(N, K, case["bias"], gen))
    # tokens of different sizes, with a few channels that are larger than the others
    x = torch.randn((M, K), generator=gen, device="cuda")
    x *= torch.rand((M, 1), generator=gen, device="cuda") * 2 + 0.2
    x *= torch.where(torch.rand((K,), generator=gen, device="cuda") < 0.02, 6.0, 1.0)
    if op == "matmul":
        state["a_scale"] = (x.abs().amax(1) / 127).clamp_min(1e-20)
        state["a"] = (x / state["a_scale"][:, None]).round().clamp(-127, 127).to(torch.int8)
    else:
        state["x"] = x.to(_TYPES[case["dtype"]])
    return state


# ---- the plain forms ---------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return torch.ones_like(z)


def _norm(x, weight, bias, groups, act):
    """(activated, mean, rstd) in 32 bits."""
    N, S, C = x.shape
    g = x.float().view(N, S, groups, C // groups)
    mean = g.mean((1, 3), keepdim=True)
    d = g - mean
    rstd = (d.square().mean((1, 3), keepdim=True) + _EPS).rsqrt()
    z = (d * rstd).view(N, S, C) * weight + bias
    return _act(z, act), mean.view(N, groups), rstd.view(N, groups)


def _norm_grad(s, groups, act):
    x, dy = s["x"].float(), s["grad"].float()
    N, S, C = x.shape
    per = C // groups
    xhat = ((x.view(N, S, groups, per) - s["mean"][:, None, :, None])
            * s["rstd"][:, None, :, None])
    z = xhat.view(N, S, C) * s["weight"] + s["bias"]
    dz = dy * _act_grad(z, act)
    d = (dz * s["weight"]).view(N, S, groups, per)
    m1 = d.mean((1, 3), keepdim=True)
    m2 = (d * xhat).mean((1, 3), keepdim=True)
    dx = (d - m1 - xhat * m2) * s["rstd"][:, None, :, None]
    return (dx.view(N, S, C).to(s["x"].dtype), (dz * xhat.view(N, S, C)).sum((0, 1)),
            dz.sum((0, 1)))


def _codes(x):
    """8-bit codes of each row, as 32-bit numbers, and the row's scale."""
    big = x.abs().amax(-1, keepdim=True)
    inverse = torch.div(torch.full_like(big, 127), big)     # a quotient, rounded once
    return (x * inverse).round(), big / 127


def _product(a, a_scale, s, act, out):
    y = (a @ s["w"].float().t()) * a_scale * s["w_scale"]
    if s["b"] is not None:
        y = y + s["b"]
    return _act(y, act).to(_TYPES[out])


def run(state):
    s = state
    c = s["case"]
    op, act = c["op"], c["act"]
    if own:
        import view_deformable_feature_amd as vdf
        if op == "norm":
            return vdf.gn_forward(s["x"], c["G"], s["weight"], s["bias"], _EPS, act)
        if op == "norm_grad":
            return vdf.gn_backward(s["x"], s["grad"], s["mean"], s["rstd"], c["G"], s["weight"],
                                   s["bias"], act)
        if op == "matmul":
            return vdf.i8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["b"],
                                 activation=act, out_dtype=_TYPES[c["out"]])
        if op == "linear":
            return vdf.i8_linear(s["x"], s["w"], s["w_scale"], s["b"], activation=act,
                                 out_dtype=_TYPES[c["out"]])
        return vdf.i8_norm_linear(s["x"], c["G"], s["weight"], s["bias"], s["w"], s["w_scale"],
                                  s["b"], eps=_EPS, activation=act, out_dtype=_TYPES[c["out"]])
    if op == "norm":
        y, mean, rstd = _norm(s["x"], s["weight"], s["bias"], c["G"], act)
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_grad":
        return _norm_grad(s, c["G"], act)
    if op == "matmul":
        return _product(s["a"].float(), s["a_scale"][:, None], s, act, c["out"])
    if op == "linear":
        a, scale = _codes(s["x"].float())
        return _product(a, scale, s, act, c["out"])
    y, _, _ = _norm(s["x"], s["weight"], s["bias"], c["G"], act)
    a, scale = _codes(y)
    # rows that an activation leaves empty have no magnitude to divide by
    a, scale = torch.where(scale > 0, a, 0.0), torch.where(scale > 0, scale, 0.0)
    N, S, C = a.shape
    y = _product(a.view(N * S, C), scale.view(N * S, 1), s, "none", c["out"])
    return y.view(N, S, c["D"])


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if op == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K + 4 * M + N * K + 4 * N + 4 * N * case["bias"]
                + M * N * size[case["out"]], "flops": 2 * M * K * N}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K * size[case["dtype"]] + N * K + 4 * N + 4 * N * case["bias"]
                + M * N * size[case["out"]], "flops": 2 * M * K * N + 4 * M * K}
    n, C, e = case["N"] * case["S"] * case["C"], case["C"], size[case["dtype"]]
    stats = 8 * case["N"] * case["G"]
    if op == "norm":
        return {"bytes": 2 * n * e + 8 * C + stats, "flops": 12 * n}
    if op == "norm_grad":
        return {"bytes": 3 * n * e + 16 * C + stats, "flops": 30 * n}
    D, rows = case["D"], case["N"] * case["S"]
    return {"bytes": n * e + 8 * C + D * C + 4 * D + 4 * D * case["bias"]
            + rows * D * size[case["out"]], "flops": 2 * n * D + 14 * n}


# ---- in 64 bits --------------------------------------------------------------------------

def _exact_act(z, act):
    if act == "relu":
        return torch.relu(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def _exact_norm(x, weight, bias, groups, act):
    """Group by group, over the values with the channel first."""
    N, S, C = x.shape
    v = x.transpose(1, 2).reshape(N, groups, (C // groups) * S)
    var, mean = torch.var_mean(v, dim=2, unbiased=False)
    r = 1 / torch.sqrt(var + _EPS)
    v = ((v - mean[..., None]) * r[..., None]).reshape(N, C, S)
    v = v * weight[None, :, None] + bias[None, :, None]
    return _exact_act(v, act).transpose(1, 2), mean, r


def _exact_codes(x):
    """The rows' codes by the definition, whose two quotients and whose product are numbers of
    32 bits (a code is a whole number: where it falls goes by them)."""
    big = x.abs().amax(-1, keepdim=True)
    full = torch.tensor(127.0, device=x.device)
    q = torch.round(x * torch.div(full, big))
    return (torch.where(big > 0, q, torch.zeros_like(q)).double(),
            torch.div(big, full).double())


def _exact_product(a, scale, s, act):
    y = torch.mm(a, s["w"].double().t().contiguous()) * (scale * s["w_scale"].double()[None, :])
    if s["b"] is not None:
        y += s["b"].double()
    return _exact_act(y, act)


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case["act"]
    if op == "matmul":
        return _exact_product(s["a"].double(), s["a_scale"].double()[:, None], s, act)
    if op == "linear":
        return _exact_product(*_exact_codes(s["x"].float()), s, act)
    x, weight, bias = (s[k].double() for k in ("x", "weight", "bias"))
    if op == "norm":
        return _exact_norm(x, weight, bias, case["G"], act)
    if op == "norm_linear":
        y = _exact_norm(x, weight, bias, case["G"], act)[0].reshape(-1, case["C"])
        big = y.abs().amax(1, keepdim=True)
        safe = torch.where(big > 0, big, torch.ones_like(big))
        q = torch.round(y * (127 / safe))
        out = _exact_product(q, big / 127, s, "none")
        return out.reshape(case["N"], case["S"], case["D"])
    for t in (x, weight, bias):
        t.requires_grad_(True)
    y, _, _ = _exact_norm(x, weight, bias, case["G"], act)
    return torch.autograd.grad(y, (x, weight, bias), s["grad"].double())
