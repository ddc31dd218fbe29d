"""The norm and the 8-bit products among the operators they stand between: a training step
through a deformable convolution and its group norm, and a serving pass whose offsets come
from 8-bit projections, eagerly and captured into a graph."""
import numpy as np
import pytest
import torch

import oracle
import view_deformable_feature_amd as vdf
from gpu_helpers import TOL_BWD, TOL_FWD, TOL_OUT_BF16, assert_close
from norm_int8_reference import Norm, check, codes, product
from test_i8_gpu import _norm_linear_ref
from view_deformable_feature_amd import workloads as W

pytestmark = pytest.mark.gpu

CONF = dict(groups=4, kernel=(3, 3), stride=(1, 1), pad=(1, 1), dilation=(1, 1))


def test_training_step_through_convolution_and_norm():
    wl = W.dcn_custom("chain", N=2, H=9, W=11, C=32, groups=4, seed=4101)
    inp = W.make_dcn_inputs(wl)
    x = torch.from_numpy(inp["input"]).cuda().requires_grad_(True)
    om = torch.from_numpy(inp["offset_mask"]).cuda().requires_grad_(True)
    w = (torch.rand(32, generator=torch.Generator().manual_seed(1)) + 0.5).cuda().requires_grad_(True)
    b = torch.randn(32, generator=torch.Generator().manual_seed(2)).cuda().requires_grad_(True)
    go = torch.from_numpy(inp["grad_out"]).cuda()
    y = vdf.deformable_conv(x, om, **CONF)
    out = vdf.group_norm_act(y, 8, w, b, activation="silu")
    (out * go).sum().backward()
    torch.cuda.synchronize()
    y_ref = oracle.dcn_forward(inp["input"], inp["offset_mask"], **CONF)
    ref = Norm(torch.from_numpy(y_ref).reshape(2, 99, 32), 8, w, b, 1e-5, "silu")
    (dy, dw, db), _ = ref.backward(go.reshape(2, 99, 32))
    gx, gom = oracle.dcn_backward(inp["input"], inp["offset_mask"],
                                  dy.reshape(2, 9, 11, 32).float().numpy(), **CONF)
    assert_close("out", out.detach().cpu().numpy().reshape(2, 99, 32), ref.y.numpy(), 5 * TOL_FWD)
    assert_close("x.grad", x.grad.cpu().numpy(), gx, TOL_BWD)
    assert_close("om.grad", om.grad.cpu().numpy(), gom, TOL_BWD)
    assert_close("w.grad", w.grad.cpu().numpy(), dw.numpy(), TOL_BWD)
    assert_close("b.grad", b.grad.cpu().numpy(), db.numpy(), TOL_BWD)


def _serving(x, layers):
    """Offsets by 8 bits, convolution, norm with activation into the next offsets, convolution."""
    (p1, s1, b1), (nw, nb), (p2, s2, b2) = layers
    N, H, Wd, C = x.shape
    y = vdf.dcn_forward_projected(x, p1, s1, b1, 4, out_dtype=torch.bfloat16)
    om = vdf.i8_norm_linear(y, 8, nw, nb, p2, s2, b2, activation="silu")
    z = vdf.dcn_forward(y, om.view(N, H, Wd, 4, 27), 4)
    return y, om, z


@pytest.mark.parametrize("C", [64, 320])
def test_serving_pass(C):
    gen = torch.Generator().manual_seed(4102)
    x = torch.randn((3, 7, 10, C), generator=gen).to(torch.bfloat16).cuda()

    def layer():
        w = torch.randn((108, C), generator=gen) * (0.6 / C ** 0.5)
        b = torch.randn(108, generator=gen) * 0.3
        return (*vdf.i8_quantize_rows(w.cuda()), b.cuda())

    layers = (layer(), ((torch.rand(C, generator=gen) + 0.5).cuda(), torch.randn(C, generator=gen).cuda()),
              layer())
    y, om, z = _serving(x, layers)
    torch.cuda.synchronize()
    # each step against its definition, from what the step before it gave
    (p1, s1, b1), (nw, nb), (p2, s2, b2) = layers
    om1 = vdf.i8_linear(x, p1, s1, b1)
    torch.cuda.synchronize()
    ref, tol = product(*codes(x.reshape(-1, C)), p1, s1, b1, "none")
    check("offsets", om1.reshape(-1, 108), ref, tol)
    bits = x.cpu().view(torch.int16).numpy().view(np.uint16)
    ref = oracle.dcn_forward(bits, om1.cpu().numpy().reshape(3, 7, 10, 4, 27), **CONF)
    assert_close("y", y.float().cpu().numpy(), ref, TOL_OUT_BF16)
    ref, tol = _norm_linear_ref(y.reshape(3, 70, C), 8, nw, nb, 1e-5, "silu", p2, s2, b2)
    check("next offsets", om.reshape(-1, 108), ref, tol)
    bits = y.cpu().view(torch.int16).numpy().view(np.uint16)
    ref = oracle.dcn_forward(bits, om.cpu().numpy().reshape(3, 7, 10, 4, 27), **CONF)
    assert_close("z", z.cpu().numpy(), ref, TOL_FWD)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _serving(x, layers)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _serving(x, layers)
    for k in range(3):
        x.mul_(1.25)
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = _serving(x, layers)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), f"replay {k}"


def test_projected_convolution_refuses():
    x = torch.zeros((1, 5, 6, 8), device="cuda")
    w = torch.zeros((108, 8), dtype=torch.int8, device="cuda")
    s = torch.zeros(108, device="cuda")
    with pytest.raises(ValueError, match="size of the input"):
        vdf.dcn_forward_projected(x, w, s, None, 4, pad=0)
    with pytest.raises(ValueError, match="54"):
        vdf.dcn_forward_projected(x, w, s, None, 2)
    with pytest.raises(ValueError, match="shape"):
        vdf.dcn_forward_projected(x[..., :4].contiguous(), w, s, None, 4)
    assert vdf.dcn_forward_projected(x[:0], w, s, None, 4).shape == (0, 5, 6, 8)


def test_norm_between_two_streams_shares_nothing():
    """Two captured graphs of the same operators, replayed at once on two streams, each with
    the workspace it was captured with."""
    xs = [torch.randn((4, 30000, 64), device="cuda") for _ in range(2)]
    graphs, outs = [], []
    for x in xs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            vdf.gn_forward(x, 8, activation="silu")
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vdf.gn_forward(x, 8, activation="silu"))
        graphs.append(g)
    want = [vdf.gn_forward(x, 8, activation="silu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, t in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, t))


@pytest.mark.parametrize("C", [64, 320])
def test_projected_convolution_into_buffers(C):
    """offset_mask, workspace and out given: nothing is allocated, the results are the same."""
    gen = torch.Generator().manual_seed(4103)
    x = torch.randn((2, 9, 12, C), generator=gen).to(torch.bfloat16).cuda()
    p, s = vdf.i8_quantize_rows((torch.randn((108, C), generator=gen) * (0.6 / C ** 0.5)).cuda())
    b = (torch.randn(108, generator=gen) * 0.3).cuda()
    want = vdf.dcn_forward_projected(x, p, s, b, 4)
    offsets = vdf.i8_linear(x, p, s, b)
    n = vdf.i8_linear_workspace_size(2 * 9 * 12, C, 108, x.dtype)
    assert (n > 0) == (C == 320)
    om = torch.full((2, 9, 12, 4, 27), float("nan"), device="cuda")
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    out = torch.full_like(want, float("nan"))
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    got = vdf.dcn_forward_projected(x, p, s, b, 4, out=out, offset_mask=om, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    torch.cuda.synchronize()
    assert got is out and torch.equal(got, want)
    assert torch.equal(om.view(2, 9, 12, 108), offsets)
    none = vdf.dcn_forward_projected(x[:0], p, s, b, 4, offset_mask=om[:0])
    assert none.shape == (0, 9, 12, C)
    with pytest.raises(ValueError, match="offset_mask has shape"):
        vdf.dcn_forward_projected(x, p, s, b, 4, offset_mask=om[..., :9].contiguous())
    with pytest.raises(TypeError, match="offset_mask has dtype"):
        vdf.dcn_forward_projected(x, p, s, b, 4, offset_mask=om.half())
    if n:
        with pytest.raises(ValueError, match="workspace"):
            vdf.dcn_forward_projected(x, p, s, b, 4, workspace=ws[:n - 1])
