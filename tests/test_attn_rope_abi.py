"""The attention's and the rotation's entry points reject malformed calls on the host before any
HIP call, and the binding checks its tensors (no GPU needed).  Pointers are fake, suitably
aligned addresses: every call here fails a host-side check or asks for a size."""
import ctypes

import pytest
import torch

import view_deformable_feature_amd as vdf
from view_deformable_feature_amd import _lib
from view_deformable_feature_amd.build import build, is_stale

FAKE = 0x10000000
FAR = 0x7000000000
FARTHER, FARTHEST = 0x7100000000, 0x7200000000
vp = ctypes.c_void_p
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    if is_stale():
        build()
    return _lib.load()


def _msg(lib):
    return lib.da_last_error().decode()


def _dense(N, H, D):
    return (ctypes.c_int64 * 3)(N * H * D, H * D, D)


def _attn(**kw):
    d = dict(batch=2, queries=30, keys=50, heads=8, key_heads=4, head_dim=32, scale=0.1, dtype=0,
             flags=0, reserved=0)
    d.update(kw)
    for n, N, H in (("q", "queries", "heads"), ("k", "keys", "key_heads"), ("v", "keys", "key_heads"),
                    ("out", "queries", "heads"), ("grad", "queries", "heads")):
        d.setdefault(n + "_stride", _dense(min(d[N], 1 << 20), min(d[H], 1 << 10), d["head_dim"]))
    return _lib.AttnProblem(**d)


def _fwd(lib, p, q=FAKE, k=FAKE, v=FAKE, lens=FAKE, mask=FAKE, out=FAR, lse=FARTHER, ws=FAKE, n=1 << 60):
    return lib.attn_forward(ref(p), vp(q), vp(k), vp(v), vp(lens), vp(mask), vp(out), vp(lse), vp(ws), n,
                            None)


def _bwd(lib, p, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, go=FAKE, lens=FAKE, mask=FAKE, gq=FAR,
         gk=FARTHER, gv=FARTHEST, ws=FAKE, n=1 << 60):
    return lib.attn_backward(ref(p), vp(q), vp(k), vp(v), vp(out), vp(lse), vp(go), vp(lens), vp(mask),
                             vp(gq), vp(gk), vp(gv), vp(ws), n, None)


ATTN_BAD = [
    (dict(batch=-1), 1, ">= 0"),
    (dict(queries=-1), 1, ">= 0"),
    (dict(keys=-2), 1, ">= 0"),
    (dict(heads=0), 1, ">= 1"),
    (dict(key_heads=0), 1, ">= 1"),
    (dict(head_dim=0), 1, ">= 1"),
    (dict(key_heads=3), 1, "multiple of key_heads"),
    (dict(dtype=3), 1, "da_dtype"),
    (dict(scale=0.0), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(scale=2.0 ** 127), 1, "scale"),
    (dict(flags=1), 1, "flags"),
    (dict(reserved=1), 1, "reserved"),
    (dict(head_dim=20), 2, "multiple of 8"),
    (dict(head_dim=136), 2, "up to 128"),
    (dict(keys=1 << 30), 2, "2^30"),
    (dict(queries=1 << 30), 2, "2^31"),
    (dict(batch=1 << 30), 2, "2^31"),
    (dict(heads=1 << 20, key_heads=1 << 20), 2, "2^24"),
    (dict(queries=1 << 26, batch=1 << 20), 2, "2^45"),
    (dict(q_stride=(ctypes.c_int64 * 3)(7680, -256, 32)), 1, "negative"),
    (dict(k_stride=(ctypes.c_int64 * 3)(6400, 130, 32)), 1, "16 bytes"),
    (dict(v_stride=(ctypes.c_int64 * 3)(6400, 128, 2)), 1, "16 bytes"),
    (dict(v_stride=(ctypes.c_int64 * 3)(1 << 60, 128, 32)), 1, "16 bytes"),
    (dict(k_stride=(ctypes.c_int64 * 3)(1 << 30, 1 << 22, 32)), 2, "2^24"),
    (dict(q_stride=(ctypes.c_int64 * 3)(1 << 56, 256, 32), batch=1 << 9), 2, "2^62"),
    (dict(out_stride=(ctypes.c_int64 * 3)(7680, 256, 30)), 1, "16 bytes"),
]


@pytest.mark.parametrize("kw, code, needle", ATTN_BAD)
def test_attention_rejects_malformed_problem(lib, kw, code, needle):
    p, n = _attn(**kw), ctypes.c_size_t(0)
    assert _fwd(lib, p) == code and needle in _msg(lib)
    assert _bwd(lib, p) == code and needle in _msg(lib)
    assert lib.attn_forward_workspace_size(ref(p), ref(n)) == code
    assert lib.attn_backward_workspace_size(ref(p), ref(n)) == code


def test_attention_rejects_launches_past_32_bits(lib):
    p = _attn(batch=1 << 15, queries=1 << 22, heads=1, key_heads=1, keys=8, head_dim=8,
              **{n + "_stride": _dense(8 if n in "kv" else 1 << 22, 1, 8)
                 for n in ("q", "k", "v", "out", "grad")})
    far = 1 << 55
    assert _fwd(lib, p, out=far, lse=2 * far) == 2 and "workgroups" in _msg(lib)
    assert _bwd(lib, p, gq=far, gk=2 * far, gv=3 * far) == 2 and "workgroups" in _msg(lib)


def test_attention_rejects_pointers(lib):
    p, h = _attn(), _attn(dtype=1)
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(out=0)):
        assert _fwd(lib, p, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(lse=0), dict(go=0), dict(gk=0),
               dict(gv=0)):
        assert _bwd(lib, p, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(q=FAKE + 8), dict(k=FAKE + 4), dict(v=FAKE + 8), dict(out=FAR + 8),
               dict(lse=FARTHER + 2), dict(lens=FAKE + 2)):
        for x in (p, h):
            assert _fwd(lib, x, **kw) == 1 and "aligned" in _msg(lib)
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 8), dict(go=FAKE + 2), dict(gq=FAR + 8),
               dict(gk=FARTHER + 4), dict(gv=FARTHEST + 8), dict(lse=FAKE + 2), dict(lens=FAKE + 1)):
        assert _bwd(lib, p, **kw) == 1 and "aligned" in _msg(lib)
    # q's 61440 bytes and k's 51200 from FAKE on
    for out in (FAKE, FAKE + 61424, FAKE - 61424):
        assert _fwd(lib, p, out=out) == 1 and "overlaps" in _msg(lib)
    assert _fwd(lib, p, lse=FAKE + 16) == 1 and _fwd(lib, p, lse=FAR + 16) == 1
    assert "overlaps" in _msg(lib)
    for kw in (dict(gq=FAKE), dict(gk=FAKE + 61424), dict(gv=FAKE - 16)):
        assert _bwd(lib, p, **kw) == 1 and "overlaps" in _msg(lib)
    for kw in (dict(gq=FARTHER), dict(gk=FARTHEST - 16), dict(gv=FAR + 16)):
        assert _bwd(lib, p, **kw) == 1 and "overlap" in _msg(lib)
    for st in ((7680, 0, 32), (7680, 256, 16), (0, 256, 32)):
        assert _fwd(lib, _attn(out_stride=(ctypes.c_int64 * 3)(*st))) == 1
        assert "places of out overlap" in _msg(lib)
    bad = _attn(grad_stride=(ctypes.c_int64 * 3)(7680, 250, 32))
    assert _bwd(lib, bad) == 1 and "grad_out" in _msg(lib)
    assert lib.attn_forward(None, *[None] * 8, 0, None) == 1 and "NULL" in _msg(lib)
    assert lib.attn_backward(None, *[None] * 12, 0, None) == 1 and "NULL" in _msg(lib)
    assert lib.attn_forward_workspace_size(ref(p), None) == 1
    assert lib.attn_backward_workspace_size(ref(p), None) == 1


def _places(at, B, N, H, D, strides):
    """The addresses of a tensor's binary32 numbers, by fours."""
    return {at + 4 * (b * strides[0] + n * strides[1] + h * strides[2] + d)
            for b in range(B) for n in range(N) for h in range(H) for d in range(0, D, 4)}


def _out_beside_q(lib, q, out, Nq, H, D, B=2):
    """What the call says of q and out, (distance in bytes, strides) each; keys enough to want a
    workspace, which it does not get."""
    p = _attn(batch=B, queries=Nq, keys=40000, heads=H, key_heads=1, head_dim=D,
              q_stride=(ctypes.c_int64 * 3)(*q[1]), out_stride=(ctypes.c_int64 * 3)(*out[1]),
              k_stride=_dense(40000, 1, D), v_stride=_dense(40000, 1, D))
    assert _fwd(lib, p, q=FAR + q[0], out=FAR + out[0], lse=FARTHEST, n=0) == 1
    return _msg(lib)


@pytest.mark.parametrize("B", [1, 2])
def test_out_among_the_heads_of_one_buffer(lib, B):
    """Places of a packed tensor: token by token beside q's heads (the same buffer holds k and v, or not),
    batch entries first or tokens first, heads first."""
    N, H, D = 7, 3, 16
    row = 8 * D
    for strides, step in (((N * row, row, D), H * D), ((row, B * row, D), H * D),
                          ((2 * H * N * D, D, N * D), H * N * D), ((N * 2 * H * D, 2 * H * D, 2 * D), D)):
        for q, out in ((0, step), (step, 0)):
            assert "workspace" in _out_beside_q(lib, (4 * q, strides), (4 * out, strides), N, H, D, B)
    strides = (N * row, row, D)
    for off in (-4, 4, 16, H * D - 4, -H * D + 4, row - 4):
        assert "overlaps" in _out_beside_q(lib, (0, strides), (4 * off, strides), N, H, D, B)
    assert "overlaps" in _out_beside_q(lib, (0, strides), (4 * H * D, (N * row, row - D, D)), N, H, D, B)


def test_out_is_refused_wherever_it_shares_a_place(lib):
    """Random strides and distances against the sets of places themselves."""
    import random
    rng, shared, taken = random.Random(7), 0, 0
    for _ in range(6000):
        B, N, H, D = rng.choice([1, 2]), rng.choice([1, 2, 3]), rng.choice([1, 2]), 8
        few = [8 * rng.randint(0, 9) if rng.random() < 0.7 else 4 * rng.randint(0, 40) for _ in range(6)]
        q = few[:3]
        out = q if rng.random() < 0.6 else few[3:]
        if rng.random() < 0.5:
            rng.shuffle(q)
        at = 4 * 4 * rng.randint(-40, 40)
        mine = _places(at, B, N, H, D, out)
        msg = _out_beside_q(lib, (0, q), (at, out), N, H, D, B)
        if "places of out" in msg:
            continue
        if mine & _places(0, B, N, H, D, q):
            shared += 1
            assert "overlaps" in msg, (B, N, H, q, out, at)
        else:
            taken += "workspace" in msg
    assert shared > 300 and taken > 300, (shared, taken)


def test_attention_workspaces(lib):
    n = ctypes.c_size_t(0)
    p = _attn(queries=1, keys=40000)            # few rows: keys are split
    assert lib.attn_forward_workspace_size(ref(p), ref(n)) == 0 and n.value > 0
    assert _fwd(lib, p, ws=0) == 1 and "workspace is NULL" in _msg(lib)
    assert _fwd(lib, p, ws=FAKE + 128) == 1 and "256-byte" in _msg(lib)
    assert _fwd(lib, p, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    q = _attn()
    assert lib.attn_backward_workspace_size(ref(q), ref(n)) == 0 and n.value >= 2 * 4 * 2 * 8 * 30
    assert _bwd(lib, q, ws=0) == 1 and _bwd(lib, q, ws=FAKE + 4) == 1
    assert _bwd(lib, q, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    for kw in (dict(batch=0), dict(queries=0)):
        e = _attn(**kw)
        assert lib.attn_forward_workspace_size(ref(e), ref(n)) == 0 and n.value == 0
        assert lib.attn_forward(ref(e), *[None] * 8, 0, None) == 0
    assert lib.attn_backward(ref(_attn(batch=0)), *[None] * 12, 0, None) == 0


BIG = [dict(batch=1, queries=1 << 20, keys=600, heads=8, key_heads=8, head_dim=128, dtype=1),
       dict(batch=1, queries=1 << 20, keys=600, heads=8, key_heads=1, head_dim=128, dtype=1),
       dict(batch=1, queries=5, keys=5 << 20, heads=1, key_heads=1, head_dim=128, dtype=0),
       dict(batch=1, queries=1 << 25, keys=7, heads=32, key_heads=32, head_dim=8, dtype=2)]


@pytest.mark.parametrize("kw", BIG)
def test_attention_gradients_of_what_the_forward_takes(lib, kw):
    """Many rows or keys, one side split: neither the query nor the call refuses the sizes (both are
    asked with a workspace of nothing, which is)."""
    far, n = 1 << 55, ctypes.c_size_t(0)
    p = _attn(**kw, **{s + "_stride": _dense(8, kw["key_heads" if s in "kv" else "heads"], kw["head_dim"])
                       for s in ("q", "k", "v", "out", "grad")})
    assert lib.attn_forward_workspace_size(ref(p), ref(n)) == 0
    assert lib.attn_backward_workspace_size(ref(p), ref(n)) == 0 and n.value > 0
    assert _bwd(lib, p, gq=far, gk=2 * far, gv=3 * far, n=0) == 1
    assert f"{n.value} needed" in _msg(lib)


@pytest.mark.parametrize("kw", [dict(batch=1 << 23, heads=1, key_heads=1), dict(batch=1 << 20, heads=24, key_heads=12),
                                dict(batch=1 << 24, heads=1, key_heads=1, head_dim=128),
                                dict(batch=1 << 23, heads=4, key_heads=1, queries=8, dtype=0)])
def test_attention_of_few_rows_rejects_launches_past_32_bits(lib, kw):
    """The form for few rows has 512 threads to a workgroup in heads of up to 128 bytes, 256 in others."""
    kw = dict(dict(queries=1, keys=3, head_dim=8, dtype=1), **kw)
    far, n = 1 << 55, ctypes.c_size_t(0)
    p = _attn(**kw, **{s + "_stride": _dense(8, kw["key_heads" if s in "kv" else "heads"], kw["head_dim"])
                       for s in ("q", "k", "v", "out", "grad")})
    assert lib.attn_forward_workspace_size(ref(p), ref(n)) == 2 and "workgroups" in _msg(lib)
    assert _fwd(lib, p, out=far, lse=2 * far) == 2 and "workgroups" in _msg(lib)


def test_attention_workspace_query_refuses_what_the_call_does(lib):
    p = _attn(batch=1 << 15, queries=1 << 22, heads=1, key_heads=1, keys=8, head_dim=8,
              **{n + "_stride": _dense(8 if n in "kv" else 1 << 22, 1, 8)
                 for n in ("q", "k", "v", "out", "grad")})
    assert lib.attn_backward_workspace_size(ref(p), ref(ctypes.c_size_t(0))) == 2
    assert "workgroups" in _msg(lib)


def _rope(**kw):
    d = dict(head_dim=32, rotated=16, eps=1e-6, magnitude=1.0, layout=0, dtype=0, flags=0, reserved=0)
    d.update(kw)
    return _lib.RopeProblem(**d)


def _heads(**kw):
    d = dict(batch=2, tokens=30, heads=8, pos_stride=30, pos_type=2, reserved=0)
    d.update(kw)
    for n in ("x_stride", "y_stride"):
        d.setdefault(n, _dense(min(d["tokens"], 1 << 20), min(d["heads"], 1 << 10), 32))
    return _lib.RopeTensor(**d)


def _rot(lib, p, t, x=FAKE, pos=FAKE, f=FAKE, y=FAR):
    return lib.rope_forward(ref(p), ref(t), vp(x), vp(pos), vp(f), vp(y), None)


def _norm(lib, p, t, x=FAKE, pos=FAKE, w=FAKE, y=FAR, k=None, kx=FARTHER, ky=FARTHEST, f=FAKE):
    none = [vp(kx), vp(FAKE), vp(FAKE), vp(ky)]
    return lib.rope_norm_forward(ref(p), ref(t), vp(x), vp(pos), vp(w), vp(y),
                                 None if k is None else ref(k), *none, vp(f), None)


def _ngrad(lib, p, t, x=FAKE, pos=FAKE, w=FAKE, g=FAKE, dx=FAR, dw=FAKE, f=FAKE, ws=FAKE, n=1 << 40):
    return lib.rope_norm_backward(ref(p), ref(t), vp(x), vp(pos), vp(w), vp(g), vp(dx), vp(dw),
                                  None, *[None] * 6, vp(f), vp(ws), n, None)


ROPE_BAD = [
    (dict(head_dim=0), 1, "head_dim"),
    (dict(rotated=17), 1, "even"),
    (dict(rotated=34), 1, "within"),
    (dict(rotated=-2), 1, "within"),
    (dict(dtype=5), 1, "da_dtype"),
    (dict(layout=2), 1, "rope_layout"),
    (dict(magnitude=float("inf")), 1, "magnitude"),
    (dict(flags=2), 1, "flags"),
    (dict(reserved=1), 1, "reserved"),
    (dict(head_dim=514), 2, "512"),
]


@pytest.mark.parametrize("kw, code, needle", ROPE_BAD)
def test_rotation_rejects_malformed_problem(lib, kw, code, needle):
    p, t, n = _rope(**kw), _heads(), ctypes.c_size_t(0)
    for f in (_rot, _norm, _ngrad):
        assert f(lib, p, t) == code and needle in _msg(lib)
    assert lib.rope_norm_backward_workspace_size(ref(p), ref(t), None, ref(n)) == code


TENSOR_BAD = [
    (dict(batch=-1), 1, ">= 0"),
    (dict(tokens=-1), 1, ">= 0"),
    (dict(heads=0), 1, ">= 1"),
    (dict(pos_type=4), 1, "pos_type"),
    (dict(pos_stride=-1), 1, "pos_stride"),
    (dict(reserved=1), 1, "reserved"),
    (dict(x_stride=(ctypes.c_int64 * 3)(1, -1, 1)), 1, "stride"),
    (dict(y_stride=(ctypes.c_int64 * 3)(1 << 57, 1, 1)), 1, "stride"),
    (dict(batch=1 << 31), 2, "2^31"),
    (dict(tokens=1 << 31), 2, "2^31"),
    (dict(heads=1 << 31), 2, "2^31"),
    (dict(batch=1 << 16, tokens=1 << 15), 2, "2^31"),
    (dict(tokens=1 << 29, heads=1 << 30), 2, "2^56"),
    (dict(x_stride=(ctypes.c_int64 * 3)(1 << 55, 256, 32), batch=1 << 9), 2, "2^62"),
]


@pytest.mark.parametrize("kw, code, needle", TENSOR_BAD)
def test_rotation_rejects_malformed_tensor(lib, kw, code, needle):
    p, t, n = _rope(), _heads(**kw), ctypes.c_size_t(0)
    for f in (_rot, _norm, _ngrad):
        assert f(lib, p, t) == code and needle in _msg(lib)
    assert _norm(lib, p, _heads(), k=t) == code
    assert lib.rope_norm_backward_workspace_size(ref(p), ref(t), None, ref(n)) == code


def test_rotation_rejects_pointers(lib):
    p, t = _rope(), _heads()
    for kw in (dict(x=0), dict(y=0), dict(f=0), dict(pos=0)):
        assert _rot(lib, p, t, **kw) == 1 and "NULL" in _msg(lib)
        assert _norm(lib, p, t, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(x=0), dict(g=0), dict(f=0), dict(pos=0)):
        assert _ngrad(lib, p, t, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(x=FAKE + 2), dict(y=FAR + 1), dict(f=FAKE + 4), dict(pos=FAKE + 4)):
        assert _rot(lib, p, t, **kw) == 1 and "aligned" in _msg(lib)
        assert _norm(lib, p, t, **kw) == 1 and "aligned" in _msg(lib)
    assert _norm(lib, p, t, w=FAKE + 2) == 1 and "aligned" in _msg(lib)
    for kw in (dict(dx=FAR + 2), dict(w=FAKE + 2), dict(dw=FAKE + 1), dict(g=FAKE + 2)):
        assert _ngrad(lib, p, t, **kw) == 1 and "aligned" in _msg(lib)
    # a result beside x but not x, x itself with other strides, and places written twice
    assert _rot(lib, p, t, y=FAKE + 64) == 1 and "overlaps" in _msg(lib)
    other = _heads(y_stride=(ctypes.c_int64 * 3)(7680, 32, 960))
    assert _rot(lib, p, other, y=FAKE) == 1 and "overlaps" in _msg(lib)
    for s in ((7680, 0, 32), (7680, 256, 16), (256, 256, 32), (100, 256, 32)):
        twice = _heads(y_stride=(ctypes.c_int64 * 3)(*s))
        assert _rot(lib, p, twice) == 1 and "overlap" in _msg(lib)
        assert _norm(lib, p, twice) == 1
    # q's result over k, k's result over q's
    k = _heads(heads=4)
    assert _norm(lib, p, t, k=k, y=FARTHER) == 1 and "overlaps" in _msg(lib)
    assert _norm(lib, p, t, k=k, ky=FAKE) == 1 and "overlaps" in _msg(lib)
    assert _norm(lib, p, t, k=k, ky=FAR + 4096) == 1 and "overlaps" in _msg(lib)
    assert _norm(lib, _rope(eps=-1.0), t) == 1 and "eps" in _msg(lib)
    assert _norm(lib, _rope(flags=1), t) == 1 and "flags" in _msg(lib)
    assert _ngrad(lib, p, t, dx=FAKE, g=FARTHER) == 1 and "overlaps" in _msg(lib)
    assert _ngrad(lib, p, t, g=FARTHER, dx=FARTHER + 64) == 1 and "overlaps" in _msg(lib)
    assert lib.rope_forward(ref(p), None, *[None] * 5) == 1
    assert lib.rope_forward(None, ref(t), *[None] * 5) == 1
    assert lib.rope_forward(ref(p), ref(_heads(batch=0)), *[None] * 5) == 0
    assert lib.rope_norm_forward(ref(p), None, *[None] * 4, None, *[None] * 4, None, None) == 0
    big = _heads(batch=1 << 10, tokens=1 << 20, heads=8)
    assert _rot(lib, p, big, y=1 << 55) == 2 and "workgroups" in _msg(lib)


def test_rotation_workspaces(lib):
    p, t, n = _rope(), _heads(), ctypes.c_size_t(0)
    assert lib.rope_norm_backward_workspace_size(ref(p), ref(t), None, ref(n)) == 0 and n.value > 0
    assert _ngrad(lib, p, t, ws=0) == 1 and "workspace is NULL" in _msg(lib)
    assert _ngrad(lib, p, t, ws=FAKE + 16) == 1 and "256-byte" in _msg(lib)
    assert _ngrad(lib, p, t, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    assert lib.rope_norm_backward_workspace_size(ref(p), ref(t), None, None) == 1


def test_binding_refuses():
    """Types, shapes, devices and names, before the library is called."""
    q, k = torch.zeros((2, 5, 4, 8)), torch.zeros((2, 7, 2, 8))
    f = torch.zeros(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="GPU"):
        vdf.attn_forward(q, k, k)
    with pytest.raises(ValueError, match="head_dim"):
        vdf.attn_forward(q[0], k, k)
    with pytest.raises(ValueError, match="fit together"):
        vdf.attn_forward(q, k, k[:, :6])
    with pytest.raises(ValueError, match="fit together"):
        vdf.attn_forward(q[:1], k, k)
    with pytest.raises(TypeError):
        vdf.attn_forward(q.double(), k.double(), k.double())
    with pytest.raises(_lib.DAError, match="scale"):
        vdf.attn_forward(q, k, k, scale=0.0)
    with pytest.raises(_lib.DAError, match="multiple of key_heads"):
        vdf.attn_workspace_size(q[:, :, :3], k, k)
    with pytest.raises(_lib.DAError, match="16 bytes"):
        vdf.attn_workspace_size(q[..., :8], torch.zeros((2, 7, 2, 9))[..., :8],
                                torch.zeros((2, 7, 2, 9))[..., :8])
    assert vdf.attn_workspace_size(q, k, k) == 0 and vdf.attn_backward_workspace_size(q, k, k) > 0
    with pytest.raises(ValueError, match="GPU"):
        vdf.attn_backward(q, k, k, q, q, q)
    with pytest.raises(ValueError, match="GPU"):
        vdf.rope_forward(q, f)
    with pytest.raises(ValueError, match="head_dim"):
        vdf.rope_forward(q[0], f)
    with pytest.raises(TypeError):
        vdf.rope_forward(q.double(), f)
    with pytest.raises(ValueError, match="GPU"):
        vdf.rope_norm_forward(q, k, None, None, f)
    with pytest.raises(ValueError, match="one type"):
        vdf.rope_norm_forward(q, k.half(), None, None, f)
    with pytest.raises(ValueError, match="grad_q_out"):
        vdf.rope_norm_backward(q, None, q[:1], None, None, None, f)
    assert vdf.rope_norm_backward_workspace_size(q, k) > 0
    for kw in (dict(rotated=7), dict(base=1.0), dict(factor=0.5), dict(scaling="cubic"),
               dict(scaling="blend"), dict(scaling="blend", trained=100, fast=1, slow=2)):
        with pytest.raises(ValueError):
            vdf.rope_frequencies(**dict(dict(rotated=8, device="cpu"), **kw))


def test_frequencies():
    """Each kind of scaling by its definition."""
    def make(**kw):
        return vdf.rope_frequencies(64, device="cpu", **kw)

    plain, one = make()
    i = torch.arange(32, dtype=torch.float64)
    assert one == 1 and torch.equal(plain, 10000.0 ** (-i / 32))
    assert torch.equal(make(scaling="linear", factor=4.0)[0], plain / 4)
    wide = make(scaling="base", factor=8.0)[0]
    assert wide[0] == 1 and abs(float(wide[-1] * 8 / plain[-1]) - 1) < 1e-14
    blend, m = make(scaling="blend", factor=16.0, trained=4096)
    turns = 4096 * plain / (2 * torch.pi)
    assert abs(m - 1.2772588722239782) < 1e-15
    assert torch.equal(blend[turns >= 40], plain[turns >= 40])
    assert torch.allclose(blend[turns <= 0.7], plain[turns <= 0.7] / 16, rtol=1e-15)
    assert ((blend <= plain) & (blend >= plain / 16 * (1 - 1e-15))).all() and (blend.diff() < 0).all()
    assert vdf.rope_frequencies(0, device="cpu")[0].shape == (0,)
    assert vdf.rope_frequencies(2, scaling="base", factor=2.0, device="cpu")[0].tolist() == [1.0]


@pytest.mark.parametrize("trained", [3, 6, 20, 100, 512, 4096, 1 << 20])
@pytest.mark.parametrize("rotated, base", [(2, 10000.0), (64, 10000.0), (128, 500000.0)])
@pytest.mark.parametrize("fast, slow", [(32.0, 1.0), (4.0, 0.5), (40.0, 2.0)])
def test_blended_frequencies_at_both_ends(trained, rotated, base, fast, slow):
    """Pairs that turn at least `fast` times within what was trained stay, those that turn at most `slow`
    times are divided, however short that is; no pair leaves the two."""
    plain = base ** (-torch.arange(0, rotated, 2, dtype=torch.float64) / rotated)
    f, _ = vdf.rope_frequencies(rotated, base, "blend", 16.0, trained, fast, slow, device="cpu")
    turns = trained * plain / (2 * torch.pi)
    assert torch.allclose(f[turns >= fast * 1.0001], plain[turns >= fast * 1.0001], rtol=1e-15)
    assert torch.allclose(f[turns <= slow * 0.9999], plain[turns <= slow * 0.9999] / 16, rtol=1e-15)
    assert ((f <= plain * (1 + 1e-15)) & (f >= plain / 16 * (1 - 1e-15))).all()
