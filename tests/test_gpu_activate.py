"""GPU tests of the gated activation and its gradient against 64-bit definitions with bounds counted in
roundings, and of the activation straight to 8 bits against the two steps."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _fp8_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
INTER, HALVES = qm.SWIGLU_INTERLEAVED, qm.SWIGLU_HALVES


def _split(y, layout):
    y = y.double().cpu().numpy()
    I = y.shape[1] // 2
    return (y[:, :I], y[:, I:]) if layout == HALVES else (y[:, 0::2], y[:, 1::2])


def _near(got, want, err, dtype):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    tol = err + ref.HALF_STEP[dtype] * (np.abs(want) + err) + ref.HALF_MIN[dtype]
    inside = np.abs(want) + tol < torch.finfo(dtype).max
    assert inside.mean() > 0.9
    bad = inside & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (got[bad][:4], want[bad][:4], tol[bad][:4])


def _check(y, grad, act, layout, **kw):
    dtype = y.dtype
    g, u = _split(y, layout)
    p = dict(alpha=kw.get("activation_alpha", 1.0), beta=kw.get("activation_beta", 0.0), limit=kw.get("swiglu_limit", math.inf))
    out = qm.activate(y, activation=act, swiglu_fusion=layout, **kw)
    assert out.dtype == dtype and out.shape == g.shape
    want, err = ref.activate(g, u, act == qm.ACT_GEGLU, **p)
    _near(out, want, err, dtype)
    gy = qm.activate_backward(grad, y, activation=act, swiglu_fusion=layout, **kw)
    assert gy.dtype == dtype and gy.shape == y.shape
    to_gate, eg, to_up, eu = ref.activate_grad(grad.double().cpu().numpy(), g, u, act == qm.ACT_GEGLU, **p)
    got_gate, got_up = _split(gy, layout)
    _near(got_gate, to_gate, eg, dtype)
    _near(got_up, to_up, eu, dtype)
    return out, gy


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("layout", [INTER, HALVES])
@pytest.mark.parametrize("act", [qm.ACT_SWIGLU, qm.ACT_GEGLU])
@pytest.mark.parametrize("rows,I", [(1, 1), (3, 7), (2, 8), (5, 9), (17, 130), (1, 2048), (300, 96), (33, 1001)])
def test_activation_and_gradient(rows, I, act, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * I)
    y = (torch.randn(rows, 2 * I, generator=g, device="cuda") * 3).to(dtype)
    grad = torch.randn(rows, I, generator=g, device="cuda").to(dtype)
    _check(y, grad, act, layout)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("act", [qm.ACT_SWIGLU, qm.ACT_GEGLU])
def test_the_whole_range_of_gates(act, dtype):
    # from 2^-20 to the type's largest, both signs, beside small and large linear parts
    top = 15 if dtype == F16 else 40
    m = torch.cat([torch.exp2(torch.linspace(-20, top, 700)), torch.linspace(0, 24, 600)])
    gate = torch.cat([m, -m]).to(dtype)
    up = torch.tensor([1.0, -0.3, 2.0 ** -10])[torch.arange(gate.numel()) % 3].to(dtype)
    y = torch.stack((gate, up), 1).reshape(13, -1).contiguous().cuda()
    grad = torch.ones(13, y.shape[1] // 2, device="cuda").to(dtype)
    _check(y, grad, act, INTER)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("layout", [INTER, HALVES])
@pytest.mark.parametrize("kw", [dict(activation_alpha=1.702, activation_beta=1.0, swiglu_limit=7.0),
                                dict(activation_alpha=0.5, swiglu_limit=0.25), dict(activation_beta=-2.0)])
def test_parameters(kw, layout, dtype):
    y = (torch.randn(40, 300, device="cuda") * 6).to(dtype)
    limit = kw.get("swiglu_limit")
    if limit:
        y[0, :50] = limit
        y[1, :50] = -limit
        y[2, :50] = 100.0
        y[3, :50] = -100.0
    _, gy = _check(y, torch.randn(40, 150, device="cuda").to(dtype), qm.ACT_SWIGLU, layout, **kw)
    if limit:
        assert gy[2, :50].eq(0).all()       # cut on both sides
        assert gy[0, :50].ne(0).float().mean() > 0.9  # at the limit itself the gradient passes
    geglu = dict(activation=qm.ACT_GEGLU, swiglu_fusion=layout)
    assert torch.equal(qm.activate(y, **geglu, **kw), qm.activate(y, **geglu))  # which takes no parameters


@pytest.mark.parametrize("act", [qm.ACT_SWIGLU, qm.ACT_GEGLU])
def test_nan_and_infinities(act):
    y = torch.ones(2, 32, device="cuda")
    y[0, 0], y[0, 3], y[0, 4], y[0, 7] = NAN, NAN, INF, INF
    out = qm.activate(y, activation=act)
    assert out[0, :2].isnan().all() and out[0, 2:4].eq(INF).all() and out[0, 4:].isfinite().all() and out[1].isfinite().all()
    assert qm.activate(y, activation=act, swiglu_limit=2.0)[0, 0].isnan()
    gy = qm.activate_backward(torch.ones(2, 16, device="cuda"), y, activation=act)
    assert gy[0, :2].isnan().all() and gy[0, 2].isnan() and gy[0, 8:].isfinite().all()
    # gates where s is 0 or 1 leave finite gradients, also where g^3 leaves the range
    big = torch.tensor([[1e38, 1.0, -1e38, 1.0, 1e13, 1.0, -1e13, 1.0]], device="cuda")
    gy = qm.activate_backward(torch.ones(1, 4, device="cuda"), big, activation=act)
    assert gy.isfinite().all() and gy[0, 0] == 1 and gy[0, 2] == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", [INTER, HALVES])
@pytest.mark.parametrize("act", [qm.ACT_SWIGLU, qm.ACT_GEGLU])
def test_gradients_whose_factors_leave_the_range_of_float32(act, layout, dtype):
    # the gradient times the linear part is more than float32 holds, and the gate's slope brings it back
    g = torch.Generator().manual_seed(9)
    low, high = (-80.0, -30.0) if act == qm.ACT_SWIGLU else (-9.0, -6.5)
    gate = torch.rand(24, 40, generator=g) * (high - low) + low
    gate[0, :8] = -200.0  # a slope of 0
    gate[1, :8] = -1e30
    sign = torch.randint(0, 2, (2, 24, 40), generator=g) * 2 - 1
    up = torch.exp2(60 + 10 * torch.rand(24, 40, generator=g)) * sign[0]
    grad = (torch.exp2(68 + 10 * torch.rand(24, 40, generator=g)) * sign[1]).to(dtype)
    y = torch.cat((gate, up), 1) if layout == HALVES else torch.stack((gate, up), 2).flatten(1)
    _, gy = _check(y.to(dtype).cuda(), grad.cuda(), act, layout)
    assert gy.isfinite().all() and not _split(gy, layout)[0][:2, :8].any()
    gy = qm.activate_backward(torch.full_like(grad, INF).cuda(), y.to(dtype).cuda(), activation=act, swiglu_fusion=layout)
    assert not np.isfinite(_split(gy, layout)[0]).any()  # what is not finite stays so


@pytest.mark.parametrize("act", [qm.ACT_SWIGLU, qm.ACT_GEGLU])
def test_gradient_against_differences(act):
    g = torch.Generator().manual_seed(4)
    y = torch.randn(8, 64, generator=g, dtype=torch.float64)
    d = torch.randn(8, 32, generator=g, dtype=torch.float64)
    y32, d32 = y.float(), d.float()
    gy = qm.activate_backward(d32.cuda(), y32.cuda(), activation=act).double().cpu()
    h = 2.0 ** -10  # third derivatives are below 3 here: h^2 / 6 of them is left
    for col in range(0, 64, 5):
        side = []
        for step in (h, -h):
            x = y32.double().clone()
            x[:, col] += step
            v, _ = ref.activate(x[:, 0::2].numpy(), x[:, 1::2].numpy(), act == qm.ACT_GEGLU)
            side.append((torch.from_numpy(v) * d32.double()).sum(1))
        want = (side[0] - side[1]) / (2 * h)
        assert bool(((gy[:, col] - want).abs() <= 4 * h * h * (1 + d32.double().abs().sum(1)) + 1e-6).all())


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("layout", [INTER, HALVES])
@pytest.mark.parametrize("rows,I", [(1, 16), (3, 128), (17, 144), (40, 1008), (5, 2048)])
def test_straight_to_8_bits(rows, I, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + I)
    y = (torch.randn(rows, 2 * I, generator=g, device="cuda") * 2).to(dtype)
    y[0] = 0
    for act in (qm.ACT_SWIGLU, qm.ACT_GEGLU):
        codes, scales = qm.activate_fp8(y, activation=act, swiglu_fusion=layout)
        # float32 inputs hold the others exactly: the same values, then the same conversion
        c, s = qm.fp8_quantize(qm.activate(y.float(), activation=act, swiglu_fusion=layout))
        assert torch.equal(codes.view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales, s)


def test_row_strides_outputs_streams_and_graph_replays():
    wide = torch.randn(50, 600, device="cuda").to(BF16)
    y, grad = wide[:, 4:260], wide[:, 300:428]
    dense_y, dense_g = y.contiguous(), grad.contiguous()
    for layout in (INTER, HALVES):
        a = qm.activate(y, swiglu_fusion=layout)
        assert torch.equal(a, qm.activate(dense_y, swiglu_fusion=layout))
        assert torch.equal(qm.activate_backward(grad, y, swiglu_fusion=layout), qm.activate_backward(dense_g, dense_y, swiglu_fusion=layout))
        c, s = qm.activate_fp8(y, swiglu_fusion=layout)
        c2, s2 = qm.activate_fp8(dense_y, swiglu_fusion=layout)
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)
    out = torch.empty(50, 128, device="cuda", dtype=BF16)
    assert qm.activate(y, out=out) is out
    with pytest.raises(ValueError, match="overlaps y"):
        qm.activate(dense_y, out=dense_y.view(-1)[:50 * 128].view(50, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = qm.activate_backward(grad, y, stream=side)
    side.synchronize()
    assert torch.equal(other, qm.activate_backward(grad, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = (qm.activate(y), *qm.activate_fp8(y), qm.activate_backward(grad, y))
    for _ in range(3):
        wide.copy_(torch.randn(50, 600, device="cuda").to(BF16))
        want = (qm.activate(y), *qm.activate_fp8(y), qm.activate_backward(grad, y))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(captured, want))


def test_no_rows_and_wrong_tensors():
    y = torch.zeros(0, 64, device="cuda")
    assert qm.activate(y).shape == (0, 32) and qm.activate_backward(y[:, :32], y).shape == (0, 64)
    assert qm.activate_fp8(y)[1].shape == (0, 1)
    y = torch.zeros(4, 64, device="cuda")
    for call in (lambda: qm.activate(y[:, :63]), lambda: qm.activate(y.double()), lambda: qm.activate(y[0]),
                 lambda: qm.activate_backward(y, y), lambda: qm.activate_backward(y[:3, :32], y),
                 lambda: qm.activate_backward(y[:, :32].half(), y), lambda: qm.activate(y, out=y[:, :31])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.activate_fp8(y[:, :40]), lambda: qm.activate(y, swiglu_fusion=qm.SWIGLU_SEPARATE),
                 lambda: qm.activate(y, swiglu_limit=-1.0), lambda: qm.activate(y, activation=3)):
        with pytest.raises(qm.QMoEError):
            call()
