"""GPU tests of one step through 8-bit experts: routing by scores, sort, products, activation and the way back,
with every gradient back to the tokens and the router's logits; step by step, against differences, captured."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as sort_ref
from tests import _fp8_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
ROUTE = dict(score=qm.SCORE_SIGMOID, scale=1.5)


class Path:
    """One layer on 8-bit experts and its gradients to the tokens and to the logits; keeps each step."""

    def __init__(self, g, H, I, E, k):
        self.E, self.k = E, k
        m1 = torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5
        m2 = torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5
        self.bias = torch.randn(E, generator=g, device="cuda") * 0.1
        self.w1, self.w2 = qm.fp8_quantize_weights(m1), qm.fp8_quantize_weights(m2)
        self.w1t, self.w2t = qm.fp8_quantize_weights(m1, transpose=True), qm.fp8_quantize_weights(m2, transpose=True)

    def __call__(self, x, logits, grad):
        s = self.__dict__
        s["ids"], s["weights"] = qm.route_scores(logits, self.k, bias=self.bias, n_groups=2, top_groups=1, group_top=2, **ROUTE)
        _, s["offsets"], s["order"], s["rr"] = qm.permute(None, self.ids, self.E)
        s["xq"] = qm.fp8_quantize(x)
        s["y"] = qm.fp8_matmul(*self.xq, *self.w1, self.offsets, sorted_routes=self.order, top_k=self.k, dtype=x.dtype)
        s["aq"] = qm.activate_fp8(self.y)
        s["rows"] = qm.fp8_matmul(*self.aq, *self.w2, self.offsets, dtype=x.dtype)
        s["out"] = qm.unpermute(self.rows, self.rr, self.weights)
        s["grad_rows"], s["grad_weights"] = qm.unpermute_backward(grad, self.rows, self.rr, self.weights)
        s["gq"] = qm.fp8_quantize(self.grad_rows)
        s["grad_act"] = qm.fp8_matmul(*self.gq, *self.w2t, self.offsets, dtype=x.dtype)
        s["grad_y"] = qm.activate_backward(self.grad_act, self.y)
        s["yq"] = qm.fp8_quantize(self.grad_y)
        s["grad_sorted"] = qm.fp8_matmul(*self.yq, *self.w1t, self.offsets, dtype=x.dtype)
        s["grad_x"] = qm.permute_backward(self.grad_sorted, self.rr)
        s["grad_logits"] = qm.route_scores_backward(self.grad_weights, logits, self.ids, **ROUTE)
        return self.out, self.weights, self.grad_x, self.grad_logits


def _inputs(g, T, H, E, dtype, padded):
    x, grad = (torch.randn(T, H, generator=g, device="cuda").to(dtype) for _ in range(2))
    logits = torch.randn(T, E, generator=g, device="cuda")
    return x, torch.where(torch.rand(T, 1, generator=g, device="cuda") < padded, -float("inf"), logits), grad


@pytest.mark.parametrize("T,padded,dtype", [(1, 0.0, BF16), (7, 0.3, F16), (300, 0.1, BF16), (301, 1.0, F16)])
def test_step_by_step(T, padded, dtype):
    H, I, E, k = 160, 208, 6, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    p = Path(g, H, I, E, k)
    x, logits, grad = _inputs(g, T, H, E, dtype, padded)
    out, _, grad_x, grad_logits = p(x, logits, grad)
    o = p.offsets.tolist()

    def product(got, rows, w):
        (a, sa), (wc, sw) = ([v.view(torch.uint8).cpu().numpy(), f.cpu().numpy()] for v, f in (rows, w))
        for e in range(E):
            at = slice(o[e], o[e + 1])
            want, acc = ref.matmul(a[at], wc[e], sa[at], sw[e])
            tol = acc + ref.HALF_STEP[dtype] * (np.abs(want) + acc) + ref.HALF_MIN[dtype]
            assert np.all(np.abs(got[at].double().cpu().numpy() - want) <= tol)
        assert got[o[E]:].eq(0).all()

    def values(q):
        return qm.fp8_dequantize(*q, F32)

    def back(got, rows, w):
        want, mag = sort_ref.unpermute(rows.double().cpu().numpy(), p.rr.cpu().numpy(), w)
        tol = k * ref.U32 * mag + ref.HALF_STEP[dtype] * mag * 1.01 + ref.HALF_MIN[dtype]
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)

    for t in range(T):
        lt, bias = logits[t].cpu().numpy(), p.bias.cpu().numpy()
        assert p.ids[t].tolist() == ref.choose(lt, bias, k, True, 2, 1, 2).tolist()
    sorted_x = [v.view(torch.uint8)[p.order.long() // k] if v.dtype == qm.FP8_DTYPE else v[p.order.long() // k] for v in p.xq]
    product(p.y, sorted_x, p.w1)
    y = p.y.double().cpu().numpy()
    act, err = ref.activate(y[:, 0::2], y[:, 1::2], False)
    step = p.aq[1].double().cpu().numpy().repeat(128, 1)[:, :I]
    # float32's error, then half a step of e4m3
    tol = err + np.maximum(2.0 ** -4 * (np.abs(act) + err), 2.0 ** -10 * step)
    assert np.all(np.abs(values(p.aq).double().cpu().numpy() - act) <= tol)
    product(p.rows, p.aq, p.w2)
    back(out, p.rows, p.weights.double().cpu().numpy())
    product(p.grad_act, p.gq, p.w2t)
    product(p.grad_sorted, p.yq, p.w1t)
    back(grad_x, p.grad_sorted, None)
    for t in range(T):
        want, mag = ref.route_grad(logits[t].cpu().numpy(), p.ids[t].cpu().numpy(), p.grad_weights[t].cpu().numpy(), True, True, 1.5)
        tol = (2 * ref.weight_error(logits[t].cpu().numpy(), None, E) + 2 * k + 16) * ref.U32 * mag + 2.0 ** -125
        assert np.all(np.abs(grad_logits[t].double().cpu().numpy() - want) <= tol)
    if padded == 1.0:
        assert o[E] == 0 and out.eq(0).all() and grad_x.eq(0).all() and grad_logits.eq(0).all()


def test_gradient_of_the_linear_path_against_differences():
    # numbers of -2 .. 2 are their own codes, and every sum is a whole number below 2048, which float16 holds: the
    # pairing of the map with its gradient and the differences hold to the last bit
    T, H, N, E, k = 40, 272, 144, 4, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w, grad = (torch.randint(-2, 3, s, generator=g, device="cuda").to(F16) for s in ((T, H), (E, N, H), (T, N)))
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.int()
    wq, wt = qm.fp8_quantize_weights(w), qm.fp8_quantize_weights(w, transpose=True)
    assert torch.equal(qm.fp8_dequantize_weights(*wq, F16), w)
    assert torch.equal(qm.fp8_dequantize_weights(*wt, F16), w.transpose(1, 2))
    _, offsets, order, rr = qm.permute(None, ids, E)

    def loss(v):
        rows = qm.fp8_matmul(*qm.fp8_quantize(v), *wq, offsets, sorted_routes=order, top_k=k, dtype=F16)
        return float((qm.unpermute(rows, rr).double() * grad.double()).sum())

    rows = qm.unpermute_backward(grad, None, rr)[0]
    grad_x = qm.permute_backward(qm.fp8_matmul(*qm.fp8_quantize(rows), *wt, offsets, dtype=F16), rr)
    base = loss(x)
    assert base == float((x.double() * grad_x.double()).sum())
    for i in torch.randint(0, T * H, (10,), generator=g, device="cuda").tolist():
        moved = x.clone().view(-1)
        step = 1.0 if moved[i] < 2 else -1.0
        moved[i] += step
        assert loss(moved.view(T, H)) - base == step * float(grad_x.view(-1)[i])


def test_captured():
    T, H, I, E, k = 40, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    p = Path(g, H, I, E, k)
    x, logits, grad = _inputs(g, T, H, E, F16, 0.1)
    p(x, logits, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = p(x, logits, grad)
    for _ in range(4):
        for old, new in zip((x, logits, grad), _inputs(g, T, H, E, F16, 0.1)):
            old.copy_(new)
        want = [t.clone() for t in p(x, logits, grad)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_runs_do_not_differ():
    # no atomic decides an order: the same bits every time
    T, H, I, E, k = 500, 512, 256, 16, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    p = Path(g, H, I, E, k)
    inputs = _inputs(g, T, H, E, BF16, 0.05)
    first = [t.clone() for t in p(*inputs)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(p(*inputs), first))
