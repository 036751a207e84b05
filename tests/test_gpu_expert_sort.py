"""GPU tests of the sort by expert and back (permute, unpermute and their gradients) against 64-bit
definitions.  Maps and copied rows have one right answer and are compared bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def _ids(rng, T, k, E, dropped):
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    lost = rng.random((T, k)) < dropped
    ids[lost] = rng.choice([-1, E, -(2 ** 31), 2 ** 31 - 1, E + 5], int(lost.sum()))
    return ids


def _rows(rng, n, H, dtype, strided=False):
    """CPU rows and the same rows on the device, optionally as a slice of wider ones."""
    x = torch.from_numpy(rng.standard_normal((n, H), dtype=np.float32)).to(dtype)
    if not strided:
        return x, x.cuda()
    wide = torch.full((n, H + 5), float("nan"), dtype=dtype, device="cuda")
    wide[:, 3:3 + H] = x.cuda()
    return x, wide[:, 3:3 + H]


# T, H, E, k, dtype, share of dropped routes, strided hidden
PERMUTE = [
    (6, 2048, 512, 10, BF16, 0.0, False),
    (1, 64, 1, 1, F16, 0.0, False),
    (1, 1, 8, 2, F16, 0.0, False),        # one column
    (5, 7, 3, 2, BF16, 0.3, True),        # rows shorter than a vector
    (33, 8, 4, 4, F16, 0.0, True),
    (70, 3, 5, 7, F32, 0.2, True),        # float32 rows shorter than a vector; top_k above E
    (129, 1001, 60, 6, F16, 0.1, True),   # odd width: a last vector that overlaps
    (300, 129, 1024, 3, F32, 0.5, False),
    (64, 40, 16, 64, BF16, 0.0, False),   # 64 routes a token
    (9, 24, 7, 1000, F16, 0.1, False),    # more routes a token than a wavefront has lanes
    (40, 16, 4, 2, BF16, 1.0, False),     # everything dropped
    (513, 72, 8, 2, BF16, 0.05, False),
    (2100, 33, 9, 8, F16, 0.1, False),    # 16,800 routes: counted in spans
    (20000, 8, 64, 1, F16, 0.0, True),    # spans of one-route tokens
    (3000, 16, 1000, 7, F32, 0.2, False),  # spans with many experts
    (40000, 8, 5, 4, BF16, 0.1, False),   # few experts in spans
    (70000, 4, 20, 3, F16, 0.05, False),  # more than 64 routes a workgroup
    (19, 8, 31, 1024, BF16, 0.2, False),  # spans of 1024-route tokens
]


@pytest.mark.parametrize("T,H,E,k,dtype,dropped,strided", PERMUTE)
def test_permute(T, H, E, k, dtype, dropped, strided):
    rng = np.random.default_rng(T * 7 + H)
    ids = _ids(rng, T, k, E, dropped)
    x, xd = _rows(rng, T, H, dtype, strided)
    idsd = torch.from_numpy(ids).cuda()
    rows, offsets, order, route_rows = qm.permute(xd, idsd, E)
    _, o2, s2, r2 = qm.permute(None, idsd, E)
    torch.cuda.synchronize()
    ro, rs, rr = ref.sort(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(order.cpu().numpy(), rs)
    assert np.array_equal(route_rows.cpu().numpy(), rr)
    want = x[torch.from_numpy(rs // k)].clone()
    want[ro[E]:] = 0
    assert torch.equal(_bits(rows.cpu()), _bits(want))
    assert torch.equal(o2, offsets) and torch.equal(s2, order) and torch.equal(r2, route_rows)


def test_permute_skewed_to_one_expert():
    ids = torch.full((3000, 2), 4, dtype=torch.int32, device="cuda")
    x = torch.randn(3000, 16, device="cuda")
    rows, offsets, order, route_rows = qm.permute(x, ids, 8)
    assert offsets.tolist() == [0] * 5 + [6000] * 4
    assert torch.equal(order, torch.arange(6000, dtype=torch.int32, device="cuda"))
    assert torch.equal(route_rows.reshape(-1), order)
    assert torch.equal(rows, x.repeat_interleave(2, 0))


def test_permute_no_tokens():
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    rows, offsets, order, route_rows = qm.permute(torch.empty((0, 32), device="cuda"), ids, 5)
    assert offsets.tolist() == [0] * 6 and rows.shape == (0, 32) and order.numel() == 0
    assert qm.unpermute(rows, route_rows).shape == (0, 32)
    g, gw = qm.unpermute_backward(torch.empty((0, 32), device="cuda"), rows, route_rows)
    assert g.shape == (0, 32) and gw.shape == (0, 2)


def test_permute_keeps_bit_patterns():
    # NaN payloads, -0 and subnormals are copied, not computed with
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).reshape(64, 1024)
    for dtype in (F16, BF16):
        x = bits.view(dtype).cuda()
        ids = torch.arange(64, dtype=torch.int32, device="cuda").remainder(5).reshape(64, 1)
        rows, _, order, _ = qm.permute(x, ids, 5)
        assert torch.equal(_bits(rows), _bits(x)[order.long()])


# T, H, k, dtype, dropped, strided rows, weighted
BACK = [
    (8, 2048, 2, F16, 0.0, False, True),
    (1, 1, 1, F32, 0.0, False, True),
    (1, 4096, 8, BF16, 0.0, False, True),
    (3, 5, 3, BF16, 0.4, True, True),      # shorter than a vector
    (37, 1001, 6, F16, 0.1, True, True),
    (65, 130, 1, F32, 0.2, True, False),
    (50, 72, 4, BF16, 0.5, False, False),
    (20, 4100, 5, F32, 0.0, False, True),
    (9, 264, 17, F16, 0.1, False, True),   # more slots than are held at once
    (300, 64, 10, BF16, 0.0, False, True),
    (4, 16390, 3, BF16, 0.3, False, True),
]


def _setup(T, H, k, dtype, dropped, strided, seed):
    rng = np.random.default_rng(seed)
    E = 6
    ids = _ids(rng, T, k, E, dropped)
    _, _, route_rows = ref.sort(ids, E)
    rows, rows_d = _rows(rng, T * k, H, dtype, strided)
    w = rng.standard_normal((T, k), dtype=np.float32)
    return rng, route_rows, torch.from_numpy(route_rows.astype(np.int32)).cuda(), rows, rows_d, w


def _sum_bound(want, mag, terms, dtype):
    # `terms` float32 roundings of partial sums no larger than mag, then one
    # rounding of the result to the type
    acc = terms * ref.U32 * mag * (1 + terms * ref.U32)
    return acc + ref.HALF_STEP[dtype] * (np.abs(want) + acc) + ref.HALF_MIN[dtype]


@pytest.mark.parametrize("T,H,k,dtype,dropped,strided,weighted", BACK)
def test_unpermute(T, H, k, dtype, dropped, strided, weighted):
    _, rr, rrd, rows, rows_d, w = _setup(T, H, k, dtype, dropped, strided, T + H)
    wd = torch.from_numpy(w).cuda() if weighted else None
    out = qm.unpermute(rows_d, rrd, wd)
    want, mag = ref.unpermute(rows.double().numpy(), rr, w.astype(np.float64) if weighted else None)
    got = out.double().cpu().numpy()
    assert out.dtype == dtype
    assert np.all(np.abs(got - want) <= _sum_bound(want, mag, k, dtype))
    if not weighted:
        assert torch.equal(_bits(qm.permute_backward(rows_d, rrd)), _bits(out))


@pytest.mark.parametrize("T,H,k,dtype,dropped,strided,weighted", BACK)
def test_unpermute_backward(T, H, k, dtype, dropped, strided, weighted):
    rng, rr, rrd, rows, rows_d, w = _setup(T, H, k, dtype, dropped, strided, 3 * T + H)
    g, gd = _rows(rng, T, H, dtype, strided)
    wd = torch.from_numpy(w).cuda() if weighted else None
    grad_rows, grad_w = qm.unpermute_backward(gd, rows_d, rrd, wd)
    only_rows, none = qm.unpermute_backward(gd, None, rrd, wd)
    assert none is None and torch.equal(_bits(only_rows), _bits(grad_rows))
    g64, r64 = g.double().numpy(), rows.double().numpy()
    want = np.zeros((T * k, H))
    want_w, mag_w = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            if rr[t, s] >= 0:
                want[rr[t, s]] = g64[t] * (float(w[t, s]) if weighted else 1.0)
                want_w[t, s] = g64[t] @ r64[rr[t, s]]
                mag_w[t, s] = np.abs(g64[t]) @ np.abs(r64[rr[t, s]])
    got = grad_rows.double().cpu().numpy()
    # one float32 product, one rounding to the type
    assert np.all(np.abs(got - want) <= _sum_bound(want, np.abs(want), 1, dtype))
    # at most H float32 roundings of partial sums no larger than the sum of magnitudes
    assert np.all(np.abs(grad_w.double().cpu().numpy() - want_w) <= (H + 1) * ref.U32 * mag_w)


def test_back_differences():
    # the way back is linear in the rows and in the weights, so a difference over a step of any
    # size equals the gradient's product with the step up to float32 rounding
    T, H, k = 21, 77, 3
    rng, rr, rrd, rows, rows_d, w = _setup(T, H, k, F32, 0.2, False, 5)
    c, cd = _rows(rng, T, H, F32)
    d, dd = _rows(rng, T * k, H, F32)
    wd = torch.from_numpy(w).cuda()
    e = torch.from_numpy(rng.standard_normal((T, k), dtype=np.float32)).cuda()
    gr, gw = qm.unpermute_backward(cd, rows_d, rrd, wd)
    c64 = cd.double()

    def loss(r, ww):
        return float((qm.unpermute(r, rrd, ww).double() * c64).sum())

    along_rows = (loss(rows_d + dd, wd) - loss(rows_d - dd, wd)) / 2
    along_w = (loss(rows_d, wd + e) - loss(rows_d, wd - e)) / 2
    # each of the T*H outputs rounds k + 1 times (and its perturbed inputs once) against magnitudes
    # bounded by the sum of |w| |row| of its slots
    kept = torch.from_numpy(rr >= 0).cuda()
    at = torch.from_numpy(np.maximum(rr, 0)).cuda().long()
    mag = ((wd.abs() + e.abs()) * kept)[..., None].double() * (rows_d.abs() + dd.abs())[at].double()
    tol = float((mag.sum(1) * c64.abs()).sum()) * (k + 3) * ref.U32
    assert abs(along_rows - float((gr.double() * dd.double()).sum())) <= 2 * tol
    assert abs(along_w - float((gw.double() * e.double()).sum())) <= (2 + H) * tol


def test_round_trip_is_identity_and_gradients_pair():
    # permute then unpermute with weights 3/4 and 1/4 (exact products and sum) gives the
    # tokens back exactly; <permute(x), g> = <x, permute_backward(g)> for the pair of linear maps
    rng = np.random.default_rng(11)
    T, H, E, k = 130, 96, 12, 2
    ids = torch.from_numpy(_ids(rng, T, k, E, 0.0)).cuda()
    x, xd = _rows(rng, T, H, BF16)
    rows, _, _, rr = qm.permute(xd, ids, E)
    w = torch.tensor([0.75, 0.25], device="cuda").repeat(T, 1)
    assert torch.equal(qm.unpermute(rows, rr, w), xd)
    xf, g = torch.randn(T, H, device="cuda"), torch.randn(T * k, H, device="cuda")
    rows, _, _, _ = qm.permute(xf, ids, E)
    a = float((rows.double() * g.double()).sum())
    b = float((xf.double() * qm.permute_backward(g, rr).double()).sum())
    tol = float((rows.abs().double() * g.abs().double()).sum()) * k * ref.U32
    assert abs(a - b) <= tol


def test_dropped_rows_never_enter():
    # a dropped route's weight and tail row may hold anything
    rr = torch.tensor([[0, -3], [-4, 1], [-2 ** 31, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    rows = torch.full((6, 16), float("nan"), device="cuda")
    rows[0], rows[1] = 2.0, 3.0
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0], [float("nan"), 1.0]], device="cuda")
    out = qm.unpermute(rows, rr, w)
    assert out[0].eq(1.0).all() and out[1].eq(3.0).all() and out[2].eq(0.0).all()
    g = torch.ones(3, 16, device="cuda")
    grad_rows, grad_w = qm.unpermute_backward(g, rows, rr, w)
    assert grad_w.tolist() == [[32.0, 0.0], [0.0, 48.0], [0.0, 0.0]]
    assert grad_rows[0].eq(0.5).all() and grad_rows[1].eq(1.0).all()
    assert grad_rows[2].eq(0).all() and grad_rows[3].eq(0).all()


def test_infinite_and_nan_rows_follow_ieee():
    rr = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    rows = torch.zeros(2, 8, device="cuda")
    rows[0, 0], rows[0, 1], rows[1, 2] = float("inf"), float("nan"), -float("inf")
    out = qm.unpermute(rows, rr, torch.tensor([[1.0, 2.0]], device="cuda"))[0]
    assert out[0] == float("inf") and torch.isnan(out[1]) and out[2] == -float("inf")
    assert torch.isnan(qm.unpermute(rows, rr, torch.tensor([[0.0, 1.0]], device="cuda"))[0, 0])


def test_large_offsets_past_32_bits():
    # rows whose element offsets pass 2^32: 70,000 routes of 65,536 columns (9.2 GB)
    T, H, k, E = 35000, 65536, 2, 3
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    ids[-1] = torch.tensor([2, 1], dtype=torch.int32)
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[-1] = torch.arange(H, device="cuda").remainder(251).to(BF16)
    rows, offsets, _, rr = qm.permute(x, ids, E)
    assert offsets.tolist() == [0, 2 * T - 2, 2 * T - 1, 2 * T]
    assert torch.equal(rows[-1], x[-1]) and torch.equal(rows[-2], x[-1])
    assert int(rows[0].count_nonzero()) == 0
    w = torch.full((T, k), 0.5, device="cuda")
    out = qm.unpermute(rows, rr, w)
    assert torch.equal(out[-1], x[-1]) and int(out[0].count_nonzero()) == 0
    del out
    g, gw = qm.unpermute_backward(x, rows, rr, w)
    assert torch.equal(g[-1], x[-1] / 2) and gw[0].eq(0).all() and gw[-1].gt(0).all()


def test_other_stream_and_graph_replays():
    rng = np.random.default_rng(3)
    T, H, E, k = 600, 264, 10, 4
    ids = torch.from_numpy(_ids(rng, T, k, E, 0.1)).cuda()
    x = torch.randn(T, H, device="cuda").to(BF16)
    g = torch.randn(T, H, device="cuda").to(BF16)
    w = torch.rand(T, k, device="cuda")

    def chain():
        rows, offsets, order, rr = qm.permute(x, ids, E)
        out = qm.unpermute(rows, rr, w)
        grad_rows, gw = qm.unpermute_backward(g, rows, rr, w)
        return rows, offsets, order, rr, out, grad_rows, gw, qm.permute_backward(grad_rows, rr)

    eager = [t.clone() for t in chain()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = qm.permute(x, ids, E, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on_side, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for step in range(4):
        x.copy_(torch.randn(T, H, device="cuda").to(BF16))
        ids.copy_(torch.from_numpy(_ids(rng, T, k, E, 0.1)))
        want = [t.clone() for t in chain()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(captured, want)), step


def test_graph_replays_with_spans():
    rng = np.random.default_rng(4)
    ids = torch.from_numpy(_ids(rng, 9000, 2, 40, 0.05)).cuda()
    ws = torch.empty(qm.permute_workspace_size(9000, 2, 40), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    qm.permute(None, ids, 40, workspace=ws)
    with torch.cuda.graph(graph):
        captured = qm.permute(None, ids, 40, workspace=ws)
    for _ in range(3):
        ids.copy_(torch.from_numpy(_ids(rng, 9000, 2, 40, 0.05)))
        graph.replay()
        torch.cuda.synchronize()
        ro, rs, rr = ref.sort(ids.cpu().numpy(), 40)
        assert np.array_equal(captured[1].cpu().numpy(), ro)
        assert np.array_equal(captured[2].cpu().numpy(), rs)
        assert np.array_equal(captured[3].cpu().numpy(), rr)


def test_runs_repeat_bit_for_bit():
    x = torch.randn(700, 1000, device="cuda")
    ids = torch.randint(0, 30, (700, 5), device="cuda").int()
    w = torch.rand(700, 5, device="cuda")
    rows, _, _, rr = qm.permute(x, ids, 30)
    first = qm.unpermute_backward(x, rows, rr, w)
    for _ in range(3):
        again = qm.unpermute_backward(x, rows, rr, w)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
