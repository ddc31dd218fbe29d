"""The group norm's and the 8-bit products' entry points reject malformed calls on the host
before any HIP call, and the binding checks its tensors (no GPU needed).  Pointers are fake,
suitably aligned addresses: every call here fails a host-side check or asks for a size."""
import ctypes

import pytest
import torch

import view_deformable_feature_amd as vdf
from view_deformable_feature_amd import _lib
from view_deformable_feature_amd.build import build, is_stale

FAKE = 0x10000000
FAR = 0x7000000000
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if is_stale():
        build()
    return _lib.load()


def _msg(lib):
    return lib.da_last_error().decode()


def _gn(**kw):
    d = dict(batch=2, rows=30, channels=32, groups=4, eps=1e-5, activation=2, x_dtype=0,
             out_dtype=0, flags=0, reserved=0)
    d.update(kw)
    return _lib.GNProblem(**d)


def _i8(**kw):
    d = dict(rows=30, in_channels=32, out_channels=24, activation=0, x_dtype=0, out_dtype=0, flags=0)
    d.update(kw)
    return _lib.I8Problem(**d)


def _gn_fwd(lib, p, x=FAKE, w=FAKE, b=FAKE, out=FAR, mean=FAKE, rstd=FAKE, ws=FAKE, n=1 << 40):
    return lib.gn_forward(ctypes.byref(p), vp(x), vp(w), vp(b), vp(out), vp(mean), vp(rstd), vp(ws),
                          n, None)


def _gn_bwd(lib, p, x=FAKE, go=FAKE, mean=FAKE, rstd=FAKE, w=FAKE, b=FAKE, gx=FAR, gw=FAKE, gb=FAKE,
            ws=FAKE, n=1 << 40):
    return lib.gn_backward(ctypes.byref(p), vp(x), vp(go), vp(mean), vp(rstd), vp(w), vp(b), vp(gx),
                           vp(gw), vp(gb), vp(ws), n, None)


def _mm(lib, p, a=FAKE, s=FAKE, w=FAKE, ws_=FAKE, b=FAKE, out=FAR, ws=FAKE, n=1 << 40):
    return lib.i8_matmul(ctypes.byref(p), vp(a), vp(s), vp(w), vp(ws_), vp(b), vp(out), vp(ws), n, None)


def _lin(lib, p, x=FAKE, w=FAKE, ws_=FAKE, b=FAKE, out=FAR, ws=FAKE, n=1 << 40):
    return lib.i8_linear(ctypes.byref(p), vp(x), vp(w), vp(ws_), vp(b), vp(out), vp(ws), n, None)


def _nl(lib, p, D=24, x=FAKE, w=FAKE, ws_=FAKE, b=FAKE, out=FAR, ws=FAKE, n=1 << 40, nw=FAKE):
    return lib.i8_norm_linear(ctypes.byref(p), D, vp(x), vp(nw), vp(FAKE), vp(w), vp(ws_), vp(b),
                              vp(out), vp(ws), n, None)


GN_BAD = [
    (dict(channels=30), 1, "multiple of groups"),
    (dict(groups=0), 1, ">= 1"),
    (dict(rows=0), 1, ">= 1"),
    (dict(channels=0), 1, ">= 1"),
    (dict(batch=-1), 1, "batch"),
    (dict(eps=-1e-5), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"),
    (dict(eps=float("inf")), 1, "eps"),
    (dict(activation=4), 1, "activation"),
    (dict(activation=-1), 1, "activation"),
    (dict(x_dtype=3), 1, "da_dtype"),
    (dict(out_dtype=-1), 1, "da_dtype"),
    (dict(flags=1), 1, "flags"),
    (dict(reserved=1), 1, "reserved"),
    (dict(channels=1 << 17, groups=1), 2, "2^16"),
    (dict(batch=1 << 31), 2, "2^31"),
    (dict(rows=1 << 31), 2, "2^31"),
    (dict(batch=1 << 30, rows=1 << 30), 2, "2^45"),
    (dict(batch=1 << 30, rows=1 << 12, channels=1 << 16, groups=1 << 16), 2, "workgroups"),
    (dict(batch=1 << 25, rows=1), 2, "workgroups"),
]


@pytest.mark.parametrize("kw, code, needle", GN_BAD)
def test_gn_rejects_malformed_problem(lib, kw, code, needle):
    p = _gn(**kw)
    n = ctypes.c_size_t(0)
    assert _gn_fwd(lib, p, out=1 << 62) == code
    assert needle in _msg(lib)
    assert _gn_bwd(lib, p, gx=1 << 62) == code
    if needle != "workgroups":
        assert lib.gn_forward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
        assert lib.gn_backward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert _nl(lib, p) == code


def test_gn_rejects_pointers(lib):
    p, h = _gn(), _gn(x_dtype=1, out_dtype=1)
    for kw in (dict(x=0), dict(out=0)):
        assert _gn_fwd(lib, p, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(x=0), dict(go=0), dict(mean=0), dict(rstd=0)):
        assert _gn_bwd(lib, p, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(x=FAKE + 2), dict(out=FAR + 2), dict(w=FAKE + 1), dict(b=FAKE + 2),
               dict(mean=FAKE + 2), dict(rstd=FAKE + 3)):
        assert _gn_fwd(lib, p, **kw) == 1 and "aligned" in _msg(lib)
    for kw in (dict(x=FAKE + 2), dict(go=FAKE + 1), dict(gx=FAR + 2), dict(gw=FAKE + 2),
               dict(gb=FAKE + 1), dict(mean=FAKE + 2), dict(rstd=FAKE + 2)):
        assert _gn_bwd(lib, p, **kw) == 1 and "aligned" in _msg(lib)
    assert _gn_fwd(lib, h, x=FAKE + 1) == 1 and "aligned" in _msg(lib)
    # overlap without being the same tensor
    assert _gn_fwd(lib, p, out=FAKE + 16) == 1 and "overlaps" in _msg(lib)
    assert _gn_fwd(lib, p, out=FAKE - 16) == 1 and "overlaps" in _msg(lib)
    assert _gn_fwd(lib, _gn(out_dtype=1), out=FAKE) == 1 and "overlaps" in _msg(lib)
    assert _gn_bwd(lib, p, gx=FAKE) == 1 and "overlaps" in _msg(lib)          # is x
    assert _gn_bwd(lib, p, x=FAR, gx=FAKE + 64) == 1 and "overlaps" in _msg(lib)
    assert lib.gn_forward(None, *[None] * 7, 0, None) == 1 and "NULL" in _msg(lib)
    assert lib.gn_forward_workspace_size(ctypes.byref(p), None) == 1


def test_gn_rejects_workspaces(lib):
    p, n = _gn(batch=4, rows=100000, channels=256, groups=8), ctypes.c_size_t(0)
    assert lib.gn_forward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    assert _gn_fwd(lib, p, ws=0) == 1 and "workspace is NULL" in _msg(lib)
    assert _gn_fwd(lib, p, ws=FAKE + 128) == 1 and "256-byte" in _msg(lib)
    assert _gn_fwd(lib, p, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    assert lib.gn_backward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    assert _gn_bwd(lib, p, ws=0) == 1 and _gn_bwd(lib, p, ws=FAKE + 8) == 1
    assert _gn_bwd(lib, p, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    # nothing to normalise, nothing to need
    e = _gn(batch=0)
    assert lib.gn_forward_workspace_size(ctypes.byref(e), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.gn_forward(ctypes.byref(e), *[None] * 7, 0, None) == 0


I8_BAD = [
    (dict(rows=-1), 1, "rows"),
    (dict(in_channels=0), 1, ">= 1"),
    (dict(out_channels=0), 1, ">= 1"),
    (dict(in_channels=131072), 2, "131071"),
    (dict(rows=1 << 31), 2, "2^31"),
    (dict(out_channels=1 << 31), 2, "2^31"),
    (dict(rows=(1 << 31) - 1, out_channels=1 << 20), 2, "workgroups"),
    (dict(rows=1, out_channels=1 << 24), 2, "2^24"),
    (dict(rows=1 << 26, in_channels=257, out_channels=1), 2, "workgroups"),
    (dict(activation=5), 1, "activation"),
    (dict(out_dtype=3), 1, "da_dtype"),
    (dict(x_dtype=7), 1, "da_dtype"),
    (dict(flags=2), 1, "flags"),
]


@pytest.mark.parametrize("kw, code, needle", I8_BAD)
def test_i8_rejects_malformed_problem(lib, kw, code, needle):
    p, n = _i8(**kw), ctypes.c_size_t(0)
    for f in (_mm, _lin):
        assert f(lib, p) == code
        assert needle in _msg(lib)
    assert lib.i8_matmul_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.i8_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code


def test_i8_rejects_pointers(lib):
    p = _i8()
    for kw in (dict(a=0), dict(s=0), dict(w=0), dict(ws_=0), dict(out=0)):
        assert _mm(lib, p, **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(x=0), dict(w=0), dict(ws_=0), dict(out=0)):
        assert _lin(lib, p, **kw) == 1 and "NULL" in _msg(lib)
        assert _nl(lib, _gn(), **kw) == 1 and "NULL" in _msg(lib)
    for kw in (dict(s=FAKE + 2), dict(ws_=FAKE + 1), dict(b=FAKE + 2), dict(out=FAR + 2)):
        assert _mm(lib, p, **kw) == 1 and "aligned" in _msg(lib)
    for kw in (dict(x=FAKE + 2), dict(ws_=FAKE + 1), dict(b=FAKE + 2), dict(out=FAR + 2)):
        assert _lin(lib, p, **kw) == 1 and "aligned" in _msg(lib)
        assert _nl(lib, _gn(), **kw) == 1 and "aligned" in _msg(lib)
    assert _nl(lib, _gn(), nw=FAKE + 2) == 1 and "aligned" in _msg(lib)
    assert _nl(lib, _gn(batch=1 << 22, rows=1)) == 2 and "2^22" in _msg(lib)
    assert _nl(lib, _gn(batch=511, rows=1), D=1 << 22) == 2 and "224" in _msg(lib)
    assert lib.i8_quantize_rows(1 << 26, 300, 0, vp(FAKE), vp(FAKE), vp(FAKE), None) == 2
    assert _nl(lib, _gn(), D=0) == 1 and "out_channels" in _msg(lib)
    assert _mm(lib, _i8(x_dtype=1)) == 1 and "x_dtype" in _msg(lib)
    assert lib.i8_quantize_rows(4, 8, 0, None, vp(FAKE), vp(FAKE), None) == 1
    assert lib.i8_quantize_rows(4, 8, 0, vp(FAKE + 2), vp(FAKE), vp(FAKE), None) == 1
    assert lib.i8_quantize_rows(4, 8, 9, vp(FAKE), vp(FAKE), vp(FAKE), None) == 1
    assert lib.i8_quantize_rows(4, 0, 0, vp(FAKE), vp(FAKE), vp(FAKE), None) == 1
    assert lib.i8_quantize_rows(-1, 8, 0, vp(FAKE), vp(FAKE), vp(FAKE), None) == 1
    assert lib.i8_quantize_rows(0, 8, 0, None, None, None, None) == 0
    assert lib.i8_matmul(None, *[None] * 7, 0, None) == 1
    assert lib.i8_matmul(ctypes.byref(_i8(rows=0)), *[None] * 7, 0, None) == 0
    assert lib.i8_linear(ctypes.byref(_i8(rows=0)), *[None] * 6, 0, None) == 0
    assert lib.i8_norm_linear(ctypes.byref(_gn(batch=0)), 8, *[None] * 8, 0, None) == 0


def test_i8_rejects_workspaces(lib):
    n = ctypes.c_size_t(0)
    p = _i8(rows=5000, in_channels=4096, out_channels=512)
    assert lib.i8_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    assert _lin(lib, p, ws=0) == 1 and "workspace is NULL" in _msg(lib)
    assert _lin(lib, p, ws=FAKE + 16) == 1 and "256-byte" in _msg(lib)
    assert _lin(lib, p, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    g = _gn(batch=4, rows=100000, channels=256, groups=8)
    assert lib.i8_norm_linear_workspace_size(ctypes.byref(g), 64, ctypes.byref(n)) == 0 and n.value > 0
    assert _nl(lib, g, ws=0) == 1 and _nl(lib, g, ws=FAKE + 4) == 1
    assert _nl(lib, g, n=n.value - 1) == 1 and str(n.value) in _msg(lib)
    assert lib.i8_linear_workspace_size(ctypes.byref(p), None) == 1
    assert lib.i8_matmul_workspace_size(ctypes.byref(p), None) == 1
    assert lib.i8_norm_linear_workspace_size(ctypes.byref(g), 64, None) == 1


def test_binding_refuses():
    """Types, shapes, devices and names, before the library is called."""
    x = torch.zeros((2, 5, 8))
    w = torch.zeros((6, 8), dtype=torch.int8)
    s = torch.ones(6)
    with pytest.raises(ValueError, match="GPU"):
        vdf.gn_forward(x, 2)
    with pytest.raises(ValueError, match="activation"):
        vdf.gn_forward(x, 2, activation="tanh")
    with pytest.raises(ValueError, match=r"\[N, ..., C\]"):
        vdf.gn_forward(x[0, 0], 2)
    with pytest.raises(TypeError):
        vdf.gn_forward(x.double(), 2)
    with pytest.raises(TypeError):
        vdf.gn_forward(x, 2, out_dtype=torch.int32)
    with pytest.raises(TypeError):
        vdf.gn_backward(x, x.double(), x, x, 2)
    with pytest.raises(ValueError, match="GPU"):
        vdf.i8_quantize_rows(x)
    with pytest.raises(ValueError, match="GPU"):
        vdf.i8_linear(x, w, s)
    with pytest.raises(ValueError, match="GPU"):
        vdf.i8_matmul(w, s, w, s)
    with pytest.raises(ValueError, match="GPU"):
        vdf.i8_norm_linear(x, 2, None, None, w, s)
    with pytest.raises(TypeError):
        vdf.i8_linear_workspace_size(4, 8, 8, torch.float64)
    with pytest.raises(_lib.DAError, match="131071"):
        vdf.i8_matmul_workspace_size(4, 1 << 20, 8)
    assert vdf.gn_workspace_size(torch.zeros((0, 5, 8)), 2) == 0


def test_result_over_an_operand_is_refused(lib):
    """out over x, the codes or w, from either side."""
    x, w, far = 0x10000000, 0x40000000, 0x70000000
    p = _i8(rows=64)      # 64 x K and N x K codes are more than 16 bytes
    for over in (x, x + 16, x - 16):
        assert _lin(lib, p, x=x, w=w, out=over) == 1 and "overlaps x" in _msg(lib)
        assert _mm(lib, _i8(rows=64, x_dtype=0), a=x, w=w, out=over) == 1
        assert "overlaps x" in _msg(lib)
        assert _nl(lib, _gn(), x=x, w=w, out=over) == 1 and "overlaps x" in _msg(lib)
        assert lib.i8_quantize_rows(64, 64, 0, vp(x), vp(over), vp(far), None) == 1
        assert "overlaps x" in _msg(lib)
    for over in (w, w + 16, w - 16):
        assert _lin(lib, p, x=x, w=w, out=over) == 1 and "overlaps w" in _msg(lib)
        assert _nl(lib, _gn(), x=x, w=w, out=over) == 1 and "overlaps w" in _msg(lib)
