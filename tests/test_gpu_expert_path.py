"""GPU tests of the sort by expert, the MXFP4 products and the way back run together, forward and back to the
tokens: every step against 64-bit sums of what it was given, the whole against differences, and captured."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _swiglu(y):
    gate, up = y[:, 0::2], y[:, 1::2]
    return gate * torch.sigmoid(gate) * up


def _swiglu_backward(y, grad):
    gate, up = y[:, 0::2], y[:, 1::2]
    s = torch.sigmoid(gate)
    return torch.stack((grad * up * s * (1 + gate * (1 - s)), grad * gate * s), 2).flatten(1)


class Path:
    """One layer on MXFP4 experts and its gradient to the tokens and to the routing weights; keeps each step."""

    def __init__(self, g, H, I, E, k):
        self.E, self.k = E, k
        m1 = torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5
        m2 = torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5
        self.w1, self.w2 = qm.mx_quantize(m1), qm.mx_quantize(m2)
        self.w1t, self.w2t = qm.mx_quantize(m1, transpose=True), qm.mx_quantize(m2, transpose=True)

    def __call__(self, x, ids, weights, grad):
        s = self.__dict__
        _, s["offsets"], s["order"], s["rr"] = qm.permute(None, ids, self.E)
        s["xq"] = qm.mx_quantize(x)
        s["y"] = qm.mx_matmul(*self.xq, *self.w1, self.offsets, sorted_routes=self.order, top_k=self.k, dtype=F32)
        s["act"] = _swiglu(self.y)
        s["aq"] = qm.mx_quantize(self.act)
        s["rows"] = qm.mx_matmul(*self.aq, *self.w2, self.offsets, dtype=x.dtype)
        s["out"] = qm.unpermute(self.rows, self.rr, weights)
        s["grad_rows"], s["grad_weights"] = qm.unpermute_backward(grad, self.rows, self.rr, weights)
        s["gq"] = qm.mx_quantize(self.grad_rows)
        s["grad_act"] = qm.mx_matmul(*self.gq, *self.w2t, self.offsets, dtype=F32)
        s["grad_y"] = _swiglu_backward(self.y, self.grad_act)
        s["yq"] = qm.mx_quantize(self.grad_y)
        s["grad_sorted"] = qm.mx_matmul(*self.yq, *self.w1t, self.offsets, dtype=x.dtype)
        s["grad_x"] = qm.permute_backward(self.grad_sorted, self.rr)
        return self.out, self.grad_weights, self.grad_x


def _ids(g, T, E, k, dropped):
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.int()
    return torch.where(torch.rand(T, k, generator=g, device="cuda") < dropped, -1, ids).contiguous()


@pytest.mark.parametrize("T,dropped,dtype", [(1, 0.0, BF16), (7, 0.3, F16), (300, 0.1, BF16), (301, 1.0, F32)])
def test_path_and_its_gradient_step_by_step(T, dropped, dtype):
    H, I, E, k = 128, 192, 6, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    p = Path(g, H, I, E, k)
    x, grad = (torch.randn(T, H, generator=g, device="cuda").to(dtype) for _ in range(2))
    ids, weights = _ids(g, T, E, k, dropped), torch.rand(T, k, generator=g, device="cuda")
    out, grad_w, grad_x = p(x, ids, weights, grad)
    o = p.offsets.tolist()

    def product(got, rows, w, dt):
        a, w = rows.double(), qm.mx_dequantize(*w, F32).double()
        for e in range(E):
            s = slice(o[e], o[e + 1])
            wt = w[e].T.contiguous()
            want, mag = a[s] @ wt, a[s].abs() @ wt.abs()
            # K truncated partial sums (2 U32 each), one rounding to the type (the 1.01: of the rounded sum)
            tol = (2 * a.shape[1] * ref.U32 + ref.HALF_STEP[dt]) * mag * 1.01 + ref.HALF_MIN[dt]
            assert bool(((got[s].double() - want).abs() <= tol).all())
        assert got[o[E]:].eq(0).all()

    def values(q):
        return qm.mx_dequantize(*q, F32)

    def back(got, rows, w):
        want, mag = ref.unpermute(rows.double().cpu().numpy(), p.rr.cpu().numpy(), w)
        tol = k * ref.U32 * mag + ref.HALF_STEP[dtype] * mag * 1.01 + ref.HALF_MIN[dtype]
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)

    product(p.y, values(p.xq)[p.order.long() // k], p.w1, F32)
    product(p.rows, values(p.aq), p.w2, dtype)
    back(out, p.rows, weights.double().cpu().numpy())
    kept = p.rr >= 0
    at = torch.where(kept, p.rr, -1 - p.rr).long()
    want = torch.where(kept[..., None], weights.double()[..., None] * grad.double()[:, None], 0.0)
    got = p.grad_rows.double()[at]
    assert bool(((got - want).abs() <= (ref.U32 + ref.HALF_STEP[dtype]) * 1.01 * want.abs() + ref.HALF_MIN[dtype]).all())
    dots = grad.double()[:, None] * p.rows.double()[at] * kept[..., None]
    assert bool(((grad_w.double() - dots.sum(-1)).abs() <= (H + 1) * ref.U32 * dots.abs().sum(-1)).all())
    product(p.grad_act, values(p.gq), p.w2t, F32)
    product(p.grad_sorted, values(p.yq), p.w1t, dtype)
    back(grad_x, p.grad_sorted, None)
    if dropped == 1.0:
        assert out.eq(0).all() and grad_x.eq(0).all() and grad_w.eq(0).all()


def _grid(g, *shape):
    """Values that any block of them holds exactly: e2m1 values, as they are at the scale of a block's largest."""
    table = torch.tensor(list(ref.E2M1) + list(-ref.E2M1), dtype=F32, device="cuda")
    return table[torch.randint(0, 16, shape, generator=g, device="cuda")]


@pytest.mark.parametrize("T,H,N,E,k", [(1, 32, 64, 1, 1), (9, 96, 160, 4, 2), (130, 256, 512, 8, 3)])
def test_gradient_of_the_linear_path_against_differences(T, H, N, E, k):
    # tokens -> sorted product -> weighted sum is linear; with e2m1 operands and powers of two as weights every
    # quantisation is exact and every sum a whole number of eighths below 2^24 of them, so the pairing of the map
    # with its gradient and the differences hold to the last bit
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w, grad = _grid(g, T, H), _grid(g, E, N, H), _grid(g, T, N)
    ids = _ids(g, T, E, k, 0.1)
    weights = torch.exp2(torch.randint(-1, 2, (T, k), generator=g, device="cuda").float())
    wq, wt = qm.mx_quantize(w), qm.mx_quantize(w, transpose=True)
    assert torch.equal(qm.mx_dequantize(*wq, F32), w) and torch.equal(qm.mx_dequantize(*wt, F32), w.transpose(1, 2))
    _, offsets, order, rr = qm.permute(None, ids, E)

    def forward(v):
        return qm.unpermute(qm.mx_matmul(*qm.mx_quantize(v), *wq, offsets, sorted_routes=order, top_k=k, dtype=F32),
                            rr, weights)

    rows = qm.unpermute_backward(grad, None, rr, weights)[0]
    grad_x = qm.permute_backward(qm.mx_matmul(*qm.mx_quantize(rows), *wt, offsets, dtype=F32), rr)

    def loss(v):
        return float((forward(v).double() * grad.double()).sum())

    base = loss(x)
    assert base == float((x.double() * grad_x.double()).sum())
    for i in torch.randint(0, T * H, (12,), generator=g, device="cuda").tolist():
        moved = x.clone().view(-1)
        step = 1.0 if moved[i] in (0.0, 1.0, 2.0, 3.0, -1.0, -2.0, -3.0, -4.0) else -float(moved[i])
        moved[i] += step
        assert loss(moved.view(T, H)) - base == step * float(grad_x.view(-1)[i])


def test_path_and_its_gradient_captured():
    T, H, I, E, k = 40, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    p = Path(g, H, I, E, k)
    x, grad = (torch.randn(T, H, generator=g, device="cuda").to(F16) for _ in range(2))
    ids, weights = _ids(g, T, E, k, 0.1), torch.rand(T, k, generator=g, device="cuda")
    p(x, ids, weights, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = p(x, ids, weights, grad)
    for _ in range(4):
        x.copy_(torch.randn(T, H, generator=g, device="cuda").to(F16))
        ids.copy_(_ids(g, T, E, k, 0.1))
        want = [t.clone() for t in p(x, ids, weights, grad)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
