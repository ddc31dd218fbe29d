"""What is measured of cross attention, its gradients, the head norm with the rotation of
positions and the rotation alone, and their plain forms.

Five operators on [batch, tokens, heads, head_dim] tensors:

* ``attn_forward``: softmax attention of queries to keys and values of another length, whose
  heads several query heads may share, with a length for each batch entry and a mask of keys;
  one query a batch entry is its serving form;
* ``attn_backward``: its gradients, from what the forward pass kept;
* ``rope_norm_forward``: queries and keys divided by their root mean square head by head,
  weighted, and rotated by the angles of their positions;
* ``rope_norm_backward``: its gradients, the weights' among them;
* ``rope_forward``: the rotation alone.

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits (angles
in 64), with ``own`` true through this package.  ``exact`` gives the same in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6


def listed():
    return [
        # one new token against the states of one sequence: latency alone
        dict(name="attn_one_token", op="attn", B=1, Nq=1, Nk=1500, H=8, Hk=8, D=64, lens="full",
             mask=False, dtype="f16"),
        # one new token for each of 16 sequences of long, different lengths, four heads to a key
        # head: the states are read once
        dict(name="attn_tokens_long", op="attn", B=16, Nq=1, Nk=16384, H=32, Hk=8, D=128,
             lens="ragged", mask=False, dtype="bf16"),
        # 900 anchors to 600 instances kept from earlier frames, some of them invalid
        dict(name="attn_900_anchors", op="attn", B=1, Nq=900, Nk=600, H=8, Hk=8, D=32, lens="full",
             mask=True, dtype="f32"),
        # long queries to longer states, bound by the matrix cores
        dict(name="attn_prompt", op="attn", B=2, Nq=4096, Nk=8192, H=16, Hk=16, D=128, lens="full",
             mask=False, dtype="bf16"),
        # a training batch of anchors and instances of different numbers
        dict(name="attn_grad_900_anchors", op="attn_grad", B=6, Nq=900, Nk=1201, H=8, Hk=8, D=64,
             lens="ragged", mask=True, dtype="f16"),
        # the gradients of a long sequence whose key heads four heads share
        dict(name="attn_grad_long", op="attn_grad", B=1, Nq=4096, Nk=4096, H=16, Hk=4, D=128,
             lens="full", mask=False, dtype="bf16"),
        # one token for each of 8 sequences
        dict(name="norm_rope_one_token", op="norm_rope", B=8, N=1, H=32, Hk=8, D=128, R=128,
             layout="half", positions="far", dtype="bf16"),
        # whole sequences
        dict(name="norm_rope_prompt", op="norm_rope", B=2, N=4096, H=32, Hk=8, D=128, R=128,
             layout="half", positions="arange", dtype="bf16"),
        # the anchors' training step, whose positions are coordinates
        dict(name="norm_rope_grad_900_anchors", op="norm_rope_grad", B=1, N=900, H=8, Hk=8, D=32,
             R=32, layout="interleaved", positions="metric", dtype="f32"),
        # whole sequences, part of each head rotated
        dict(name="norm_rope_grad_long", op="norm_rope_grad", B=2, N=4096, H=16, Hk=4, D=128, R=64,
             layout="half", positions="arange", dtype="bf16"),
        # ragged sizes, half of each head, far positions
        dict(name="rope_part_far", op="rope", B=3, N=1777, H=9, D=80, R=40, layout="interleaved",
             positions="far", dtype="f32"),
        # queries of whole sequences
        dict(name="rope_whole", op="rope", B=4, N=4096, H=32, D=128, R=128, layout="half",
             positions="arange", dtype="f16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_tokens", "attn_grad", "norm_rope", "norm_rope_grad", "rope"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    D = 8 * rng.choice([2, 3, 4, 4, 5, 6, 8, 8, 9, 10, 12, 14, 16, 16])
    Hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    H = Hk * group if Hk * group <= 32 else Hk
    if op.startswith("attn"):
        B = _spread(rng, 1, 16)
        lens, mask = rng.choice(["full", "ragged"]), rng.random() < 0.4
        c = dict(op="attn_grad" if op == "attn_grad" else "attn", B=B, H=H, Hk=Hk, D=D, lens=lens,
                 mask=mask, dtype=dtype)
        if op == "attn_tokens":
            c["Nq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
            c["Nk"] = _spread(rng, 64, max(65, min(16384, (1 << 26) // (B * Hk * D))))
            return c
        # 32 bits have a sixteenth of the matrix rate
        most = (1 << 31) if dtype != "f32" else (1 << 28)
        most = max(4096, most // (B * H * D) // (4 if op == "attn_grad" else 1) * 8)
        c["Nq"] = _spread(rng, 16, max(17, min(4096, most // 64)))
        c["Nk"] = _spread(rng, 32, max(33, min(8192, most // c["Nq"], (1 << 26) // (B * Hk * D))))
        return c
    if op == "rope":
        H, Hk = rng.choice([1, 3, 8, 9, 16, 32]), 0
    B = _spread(rng, 1, 16)
    c = dict(op=op, B=B, N=_spread(rng, 1, max(1, min(8192, (1 << 24) // (B * (H + Hk) * D)))), H=H, D=D,
             R=rng.choice([D, D, D // 2 // 2 * 2, D // 4 // 2 * 2]),
             layout=rng.choice(["half", "interleaved"]),
             positions=rng.choice(["arange", "far", "metric"]), dtype=dtype)
    if op != "rope":
        c["Hk"] = Hk
    return c


def _lengths(case):
    """The numbers of keys of the batch entries: all, or different ones (of three or more
    sequences the last has none)."""
    B, Nk = case["B"], case["Nk"]
    if case["lens"] == "full":
        return [Nk] * B
    lens = [max(1, Nk - (b * 2477) % (Nk // 2 + 1)) for b in range(B)]
    if B > 2:
        lens[-1] = 0
    return lens


def _tensor(shape, gen, dtype, spread=1.0, offset=0.0):
    """Normal numbers, with an offset of its own for each place in a head."""
    x = torch.randn(shape, generator=gen, device="cuda") * spread
    if offset:
        x += torch.randn(shape[-1:], generator=gen, device="cuda") * offset
    return x.to(_TYPES[dtype])


def _attention_state(c, gen):
    B, Nq, Nk, H, Hk, D, t = (c[k] for k in ("B", "Nq", "Nk", "H", "Hk", "D", "dtype"))
    s = dict(q=_tensor((B, Nq, H, D), gen, t, 1.4), k=_tensor((B, Nk, Hk, D), gen, t, 1.0, 0.3),
             v=_tensor((B, Nk, Hk, D), gen, t, 1.0, 0.3), lens=None, mask=None)
    if c["lens"] != "full":
        s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    if c["mask"]:
        s["mask"] = torch.rand((B, Nk), generator=gen, device="cuda") < 0.85
    if c["op"] == "attn_grad":
        s["out"], s["lse"] = _attention(s)
        s["grad"] = _tensor((B, Nq, H, D), gen, t)
    return s


def _positions(c, n, gen):
    if c["positions"] == "arange":
        return None                                     # 0, 1, 2, ...
    if c["positions"] == "far":                         # sequences that go on from somewhere
        start = torch.randint(0, 1 << 20, (c["B"], 1), generator=gen, device="cuda")
        return start + torch.arange(n, device="cuda")
    return torch.rand((c["B"], n), generator=gen, device="cuda") * 120 - 60


def _rotary_state(c, gen):
    B, N, H, D, t = (c[k] for k in ("B", "N", "H", "D", "dtype"))
    # a context of eight times the trained length: longer wavelengths are stretched
    i = torch.arange(c["R"] // 2, dtype=torch.float64, device="cuda")
    freqs = 10000.0 ** (-2 * i / c["R"])
    s = dict(freqs=torch.where(freqs < 1e-2, freqs / 8, freqs), positions=_positions(c, N, gen))
    if c["op"] == "rope":
        s["x"] = _tensor((B, N, H, D), gen, t, 1.0, 0.3)
        return s
    for name, heads in (("q", H), ("k", c["Hk"])):
        s[name] = _tensor((B, N, heads, D), gen, t, 1.5, 0.5)
        s[name + "_weight"] = torch.rand((D,), generator=gen, device="cuda") + 0.5
        if c["op"] == "norm_rope_grad":
            s["grad_" + name] = _tensor((B, N, heads, D), gen, t)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = _attention_state if case["op"].startswith("attn") else _rotary_state
    return dict(make(case, gen), case=case)


# ---- the plain forms ---------------------------------------------------------------------

def _visible(s):
    """[B, Nk], true where a key may be seen, or None."""
    see = s["mask"]
    if s["lens"] is not None:
        inside = torch.arange(s["k"].shape[1], device="cuda") < s["lens"][:, None]
        see = inside if see is None else see & inside
    return see


def _heads_first(x, Hk):
    """[B, N, H, D] to [B, Hk, (H / Hk) N, D] in 32 bits: the rows that share a key head."""
    B, N, H, D = x.shape
    x = x.float().view(B, N, Hk, H // Hk, D).permute(0, 2, 3, 1, 4)
    return x.reshape(B, Hk, (H // Hk) * N, D)


def _heads_last(x, N, H):
    B, Hk, rows, D = x.shape
    return x.view(B, Hk, H // Hk, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H, D)


def _scores(s, see):
    Hk, D = s["k"].shape[2:]
    k = _heads_first(s["k"], Hk)
    z = _heads_first(s["q"], Hk) @ k.transpose(2, 3).contiguous() * (1 / math.sqrt(D))
    return z if see is None else z.masked_fill(~see[:, None, None, :], -math.inf)


def _attention(s):
    B, Nq, H, D = s["q"].shape
    Hk = s["k"].shape[2]
    see = _visible(s)
    z = _scores(s, see)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    v = _heads_first(s["v"], Hk)
    if see is not None:
        v = v * see[:, None, :, None]
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).view(B, H, Nq)
    return _heads_last(out, Nq, H).to(s["q"].dtype), lse


def _attention_grad(s):
    B, Nq, H, D = s["q"].shape
    Hk = s["k"].shape[2]
    see = _visible(s)
    lse = s["lse"].view(B, Hk, -1, 1)
    p = torch.exp(_scores(s, see) - torch.where(lse == -math.inf, 0.0, lse))
    q, k, v, out, do = (_heads_first(s[n], Hk) for n in ("q", "k", "v", "out", "grad"))
    dv = p.transpose(2, 3).contiguous() @ do
    dz = p * (do @ v.transpose(2, 3).contiguous() - (do * out).sum(-1, keepdim=True))
    dz = dz * (1 / math.sqrt(D))
    dq, dk = dz @ k, dz.transpose(2, 3).contiguous() @ q
    t = s["q"].dtype
    return (_heads_last(dq, Nq, H).to(t), dk.transpose(1, 2).to(t).contiguous(),
            dv.transpose(1, 2).to(t).contiguous())


def _angles(s, n):
    """Cosines and sines [B or 1, n, 1, pairs], from angles in 64 bits."""
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(n, device="cuda")[None]
    t = pos.double()[:, :, None, None] * s["freqs"]
    return torch.cos(t).float(), torch.sin(t).float()


def _rotate(x, cos, sin, layout):
    R = 2 * cos.shape[-1]
    y = x.clone()
    a, b = ((x[..., 0:R:2], x[..., 1:R:2]) if layout == "interleaved"
            else (x[..., :R // 2], x[..., R // 2:R]))
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if layout == "interleaved":
        y[..., 0:R:2], y[..., 1:R:2] = ya, yb
    else:
        y[..., :R // 2], y[..., R // 2:R] = ya, yb
    return y


def _norm_rotate(x, weight, cos, sin, layout):
    v = x.float()
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
    return _rotate(v * r * weight, cos, sin, layout).to(x.dtype)


def _norm_rotate_grad(x, weight, grad, cos, sin, layout):
    v = x.float()
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
    hat = v * r
    dn = _rotate(grad.float(), cos, -sin, layout)
    g = dn * weight
    dx = r * (g - hat * (g * hat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dn * hat).sum((0, 1, 2))


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        import view_deformable_feature_amd as vdf
        if op == "attn":
            return vdf.attn_forward(s["q"], s["k"], s["v"], s["lens"], s["mask"])
        if op == "attn_grad":
            return vdf.attn_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["grad"],
                                     s["lens"], s["mask"])
        if op == "norm_rope":
            return vdf.rope_norm_forward(s["q"], s["k"], s["q_weight"], s["k_weight"], s["freqs"],
                                         s["positions"], s["positions"], _EPS, c["layout"])
        if op == "norm_rope_grad":
            return vdf.rope_norm_backward(s["q"], s["k"], s["grad_q"], s["grad_k"], s["q_weight"],
                                          s["k_weight"], s["freqs"], s["positions"], s["positions"],
                                          _EPS, c["layout"])
        return vdf.rope_forward(s["x"], s["freqs"], s["positions"], c["layout"])
    if op == "attn":
        return _attention(s)
    if op == "attn_grad":
        return _attention_grad(s)
    cos, sin = _angles(s, c["N"])
    if op == "rope":
        return _rotate(s["x"].float(), cos, sin, c["layout"]).to(s["x"].dtype)
    if op == "norm_rope":
        return (_norm_rotate(s["q"], s["q_weight"], cos, sin, c["layout"]),
                _norm_rotate(s["k"], s["k_weight"], cos, sin, c["layout"]))
    dq, dqw = _norm_rotate_grad(s["q"], s["q_weight"], s["grad_q"], cos, sin, c["layout"])
    dk, dkw = _norm_rotate_grad(s["k"], s["k_weight"], s["grad_k"], cos, sin, c["layout"])
    return dq, dk, dqw, dkw


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op.startswith("attn"):
        B, Nq, Nk, H, Hk, D = (case[k] for k in ("B", "Nq", "Nk", "H", "Hk", "D"))
        keys = sum(_lengths(case))
        rows, states = B * Nq * H, keys * Hk * D * e
        extra = 4 * B * (case["lens"] != "full") + B * Nk * case["mask"] + 4 * rows
        if op == "attn":
            return {"bytes": 2 * rows * D * e + 2 * states + extra, "flops": 4 * Nq * H * D * keys}
        return {"bytes": 4 * rows * D * e + 2 * states + 2 * B * Nk * Hk * D * e + extra,
                "flops": 10 * Nq * H * D * keys}
    B, N, D, R = (case[k] for k in ("B", "N", "D", "R"))
    n = B * N * (case["H"] + case.get("Hk", 0)) * D
    pos = {"arange": 0, "far": 8, "metric": 4}[case["positions"]] * B * N + 4 * R
    if op == "rope":
        return {"bytes": 2 * n * e + pos, "flops": 3 * n}
    if op == "norm_rope":
        return {"bytes": 2 * n * e + pos + 8 * D, "flops": 7 * n}
    return {"bytes": 3 * n * e + pos + 16 * D, "flops": 14 * n}


# ---- in 64 bits --------------------------------------------------------------------------

def _exact_entry(c, s, b, h, grads):
    """One batch entry and head: out and lse, or the gradients to q, k, v, of the visible keys."""
    hk = h // (c["H"] // c["Hk"])
    keep = torch.arange(_lengths(c)[b], device="cuda")
    if s["mask"] is not None:
        keep = keep[s["mask"][b, :len(keep)]]
    q, k, v = s["q"][b, :, h].double(), s["k"][b, keep, hk].double(), s["v"][b, keep, hk].double()
    z = torch.mm(q, k.t().contiguous()) / math.sqrt(c["D"])
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    if not grads:
        return torch.mm(p, v), lse
    do = s["grad"][b, :, h].double()
    dp = torch.mm(do, v.t().contiguous())
    dz = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["D"])
    return keep, hk, torch.mm(dz, k), torch.mm(dz.t().contiguous(), q), torch.mm(p.t().contiguous(), do)


def _exact_attention(c, s):
    B, H, Nq = c["B"], c["H"], c["Nq"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["op"] == "attn":
        out = torch.zeros(s["q"].shape, **f64)
        lse = torch.full((B, H, Nq), -math.inf, **f64)
        for b in range(B):
            for h in range(H) if _lengths(c)[b] else ():
                out[b, :, h], lse[b, h] = _exact_entry(c, s, b, h, False)
        return out, lse
    dq, dk, dv = (torch.zeros(s[n].shape, **f64) for n in ("q", "k", "v"))
    for b in range(B):
        for h in range(H):
            keep, hk, gq, gk, gv = _exact_entry(c, s, b, h, True)
            dq[b, :, h] = gq
            dk[b, keep, hk] += gk
            dv[b, keep, hk] += gv
    return dq, dk, dv


def _exact_rotary(c, s, x, weight):
    """By complex numbers; differentiable."""
    R = c["R"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device="cuda").expand(c["B"], -1)
    t = pos.double()[:, :, None, None] * s["freqs"]
    if weight is not None:
        x = x * weight / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + _EPS)
    r = x[..., :R]
    if c["layout"] == "half":
        r = r.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    else:
        r = r.unflatten(-1, (R // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(r.contiguous()) * torch.polar(torch.ones_like(t), t))
    if c["layout"] == "half":
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., R:]), -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("attn"):
        return _exact_attention(c, s)
    if c["op"] == "rope":
        return _exact_rotary(c, s, s["x"].double(), None)
    x, w = ([s[n + end].double() for n in ("q", "k")] for end in ("", "_weight"))
    if c["op"] == "norm_rope":
        return tuple(_exact_rotary(c, s, *xw) for xw in zip(x, w))
    for t in x + w:
        t.requires_grad_(True)
    y = [_exact_rotary(c, s, *xw) for xw in zip(x, w)]
    return torch.autograd.grad(y, x + w, [s["grad_q"].double(), s["grad_k"].double()])
