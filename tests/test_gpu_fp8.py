"""GPU tests of 8-bit floating point in blocks of 128: conversions bit for bit against a 64-bit definition, the
grouped product against float64 sums of the values that codes and scales stand for."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as sort_ref
from tests import _fp8_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _check_rows(x):
    codes, scales = qm.fp8_quantize(x)
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == F32
    want_c, want_s = ref.quantize(x.double().cpu().numpy().reshape(-1, x.shape[-1]), 1)
    assert np.array_equal(scales.double().cpu().numpy().reshape(want_s.shape), want_s, equal_nan=True)
    assert np.array_equal(_bytes(codes).reshape(want_c.shape), want_c)
    return codes, scales


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 112), (2, 128), (17, 144), (257, 400), (2, 14336), (5, 2048)])
def test_quantize_rows(rows, K, dtype):
    g = torch.Generator().manual_seed(rows * K)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-12, 8, (rows, 1), generator=g))
    _check_rows(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantize_every_pattern(dtype):
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    _check_rows(x.reshape(-1, 128).cuda())
    alone = torch.zeros(4096, 128, dtype=dtype)  # each as its block's largest
    alone[:, 5] = x[::16]
    alone[:, 77] = -x[::16] / 3
    _check_rows(alone.cuda())


def test_quantize_borders_and_neighbours():
    # every border between neighbouring codes, with the next float32 on both sides, at many scales
    mid = torch.from_numpy((ref.E4M3[:-1] + ref.E4M3[1:]) / 2).to(F32)
    v = torch.cat([mid, torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(0.0)), torch.from_numpy(ref.E4M3).to(F32)])
    v = torch.cat([v, -v])
    v = torch.cat([v, torch.zeros(-v.numel() % 127)]).reshape(-1, 127)
    block = torch.cat([v, torch.full((v.shape[0], 1), 448.0)], 1)
    for e in (-126, -125, -100, -1, 0, 1, 63, 119):
        _check_rows((block.double() * 2.0 ** e).to(F32).cuda())


def test_quantize_scales_at_their_borders():
    tops = [448.0, float(np.nextafter(np.float32(448), np.float32(1e9))), float(np.nextafter(np.float32(448), np.float32(0))), 256.0, 511.0, 512.0]
    rows = []
    for e in (-149, -135, -134, -126, -60, 0, 100, 118, 119):
        for t in tops:
            v = t * 2.0 ** e
            if v < 3.4e38:
                rows.append([v, -v / 2] + [v / 3] * 126)
    rows += [[0.0] * 128, [-0.0] * 128, [2.0 ** -149] + [0.0] * 127, [3.4028234663852886e38] * 128,
             [1.0] * 127 + [NAN], [INF] + [1.0] * 127, [-INF] * 128, [NAN] * 128]
    _, scales = _check_rows(torch.tensor(np.array(rows, np.float32)).cuda())
    assert scales[-4:].isnan().all() and scales[-8].item() == 2.0 ** -126


def test_quantize_leaves_other_blocks_of_a_bad_row_alone():
    x = torch.randn(3, 400, device="cuda")
    x[1, 130] = NAN
    _, scales = _check_rows(x)
    assert scales.isnan().sum() == 1 and scales[1, 1].isnan()


def test_quantize_row_stride_and_leading_dimensions():
    wide = torch.randn(37, 500, device="cuda").to(BF16)
    _check_rows(wide[:, 7:7 + 272])
    _check_rows(torch.randn(3, 5, 64, device="cuda"))
    _check_rows(torch.randn(176, device="cuda").to(F16))
    assert qm.fp8_quantize(torch.empty(0, 64, device="cuda"))[1].shape == (0, 1)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 144), (1, 257, 400), (2, 16, 256), (1, 1000, 48), (4, 112, 272)])
def test_quantize_squares_and_their_transposes(E, N, K, dtype):
    g = torch.Generator().manual_seed(N + K)
    w = (torch.randn(E, N, K, generator=g) * torch.exp2(torch.randint(-6, 6, (E, N, 1), generator=g))).to(dtype)
    w[0, 0, 3] = NAN
    codes, scales = qm.fp8_quantize_weights(w.cuda())
    for e in range(E):
        want_c, want_s = ref.quantize(w[e].double().numpy(), 128)
        assert np.array_equal(_bytes(codes[e]), want_c)
        assert np.array_equal(scales[e].double().cpu().numpy(), want_s, equal_nan=True)
    one = qm.fp8_quantize_weights(w[0].cuda())
    assert torch.equal(one[0].view(torch.uint8), codes[0].view(torch.uint8))
    # the transposed input needs only its rows in sixteens
    tc, ts = qm.fp8_quantize_weights(w.cuda().transpose(1, 2).contiguous(), transpose=True)
    assert tc.shape == codes.shape and torch.equal(tc.view(torch.uint8), codes.view(torch.uint8))
    assert torch.equal(ts.nan_to_num(7.0), scales.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_dequantize_every_code(dtype):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(40, 1)
    scales = torch.exp2(torch.arange(80, dtype=F32).reshape(40, 2) * 3 - 110)
    scales[3, 1] = NAN
    got = qm.fp8_dequantize(codes.view(torch.float8_e4m3fn).cuda(), scales.cuda(), dtype).cpu()
    # exact in float64; the type rounds it once (float32: exact within its range)
    want = torch.from_numpy(ref.values(codes.numpy(), scales.numpy())).to(F32).to(dtype)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~want.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (3, 130, 272), (2, 128, 128), (1, 700, 48)])
def test_dequantize_with_a_checkpoints_scales(E, N, K):
    rng = np.random.default_rng(N)
    codes = _finite_codes(rng, (E, N, K))
    scales = rng.uniform(0.001, 3.0, (E, -(-N // 128), -(-K // 128))).astype(np.float32)
    c, s = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda()
    for dtype in (F16, BF16, F32):
        got = qm.fp8_dequantize_weights(c, s, dtype).double().cpu().numpy()
        for e in range(E):
            want = ref.values(codes[e], scales[e], 128)
            tol = (ref.U32 + ref.HALF_STEP[dtype]) * 1.01 * np.abs(want) + ref.HALF_MIN[dtype]  # two roundings
            assert np.all(np.abs(got[e] - want) <= tol)
        assert torch.equal(qm.fp8_dequantize_weights(c[0], s[0], dtype), qm.fp8_dequantize_weights(c, s, dtype)[0])


def test_values_come_back_within_half_a_step():
    x = torch.randn(64, 400, device="cuda")
    c, s = qm.fp8_quantize(x)
    y = qm.fp8_dequantize(c, s, F32)
    step = s.repeat_interleave(128, -1)[:, :400]
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its normal values
    assert bool(((y - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, step * 2.0 ** -10)).all())
    c2, s2 = qm.fp8_quantize(y)
    assert torch.equal(qm.fp8_dequantize(c2, s2, F32), y)


# ---------------------------------------------------------------- product
def _finite_codes(rng, shape):
    c = rng.integers(0, 127, shape, dtype=np.uint8)
    return c | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)


def _matmul_case(T, k, E, K, N, dtype, gather, seed, dropped=0.0, counts=None):
    """Runs one product and compares every output; returns it."""
    rng = np.random.default_rng(seed)
    R = T * k
    if counts is None:
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        ids[rng.random((T, k)) < dropped] = -1
    else:
        ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32).reshape(T, k)
        ids[ids >= E] = -1
    offsets, order, _ = sort_ref.sort(ids, E)
    kb, nb = -(-K // 128), -(-N // 128)
    ac = _finite_codes(rng, (T if gather else R, K))
    wc = _finite_codes(rng, (E, N, K))
    # scales of any value, those of one block far from its neighbours'
    as_ = (rng.uniform(0.5, 1.0, (ac.shape[0], kb)) * 2.0 ** rng.integers(-12, -6, (ac.shape[0], kb))).astype(np.float32)
    ws = (rng.uniform(0.5, 1.0, (E, nb, kb)) * 2.0 ** rng.integers(-12, -6, (E, nb, kb))).astype(np.float32)
    dev = [torch.from_numpy(v).cuda() for v in (ac, as_, wc, ws, offsets.astype(np.int32), order.astype(np.int32))]
    dev[0], dev[2] = dev[0].view(torch.float8_e4m3fn), dev[2].view(torch.float8_e4m3fn)
    out = qm.fp8_matmul(*dev[:5], sorted_routes=dev[5] if gather else None, top_k=k, dtype=dtype)
    assert out.dtype == dtype and tuple(out.shape) == (R, N)
    if gather:
        ac, as_ = ac[order // k], as_[order // k]
    want, acc = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        if offsets[e + 1] > offsets[e]:
            sl = slice(offsets[e], offsets[e + 1])
            want[sl], acc[sl] = ref.matmul(ac[sl], wc[e], as_[sl], ws[e])
    got = out.double().cpu().numpy()
    tol = acc + ref.HALF_STEP[dtype] * (np.abs(want) + acc) + ref.HALF_MIN[dtype]
    inside = np.abs(want) + tol < torch.finfo(dtype).max
    assert inside.mean() > 0.99
    assert np.all(np.abs(got - want)[inside] <= tol[inside])
    assert np.all(got[offsets[E]:] == 0)
    return out


# T, k, E, K, N, dtype, gather, dropped
PRODUCT = [
    (1, 1, 1, 16, 1, F16, False, 0.0),        # the smallest of everything
    (1, 2, 8, 2048, 512, F16, True, 0.0),     # one token
    (1, 8, 40, 512, 96, BF16, True, 0.0),
    (6, 10, 64, 256, 200, BF16, True, 0.0),
    (5, 3, 4, 112, 33, F16, True, 0.3),       # a short block, odd N, dropped routes
    (17, 2, 3, 144, 127, F16, False, 0.2),
    (40, 2, 8, 528, 130, BF16, True, 0.0),
    (100, 1, 1, 1024, 256, F16, False, 0.0),
    (130, 3, 5, 768, 257, BF16, True, 0.1),
    (256, 2, 2, 304, 300, F16, True, 0.0),
    (300, 4, 6, 1056, 520, BF16, True, 0.05),
    (512, 1, 700, 64, 40, F16, True, 0.1),    # more experts than rows a tile
    (700, 2, 2, 256, 513, F16, False, 0.0),
    (1000, 2, 3, 2064, 264, BF16, True, 0.0),
    (1500, 1, 1, 512, 640, F16, False, 0.0),
    (9, 1, 2, 48, 5000, BF16, False, 0.5),
    (300, 1, 1, 2080, 2000, BF16, False, 0.0),
    (250, 2, 8, 2048, 1100, F16, True, 0.1),
    (120, 1, 2, 3808, 700, F16, False, 0.0),
    (33, 1, 1, 8192, 130, BF16, False, 0.0),
    (1100, 1, 4, 2112, 1600, BF16, True, 0.05),
    (1024, 1, 1, 4096, 2900, F16, False, 0.0),
    (2100, 1, 2, 640, 4100, BF16, True, 0.0),
    (2048, 1, 1, 1024, 4096, F16, False, 0.0),
]


@pytest.mark.parametrize("T,k,E,K,N,dtype,gather,dropped", PRODUCT)
def test_matmul(T, k, E, K, N, dtype, gather, dropped):
    _matmul_case(T, k, E, K, N, dtype, gather, T + K + N, dropped)


@pytest.mark.parametrize("counts", [
    [0, 0, 0, 31, 1], [32, 0, 0, 0], [1, 0, 33, 0, 30], [64, 63, 65], [0, 0, 128], [127, 129],
    [1] * 16, [0] * 9 + [16] + [0] * 6, [255, 1, 257, 0, 511], [17, 15, 0, 48, 16],
])
def test_matmul_row_counts(counts):
    _matmul_case(sum(counts), 1, len(counts), 288, 144, F16, False, 1 + len(counts), counts=counts)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_matmul_one_expert_without_offsets(rows):
    rng = np.random.default_rng(rows)
    K, N = 400, 144
    ac, wc = _finite_codes(rng, (rows, K)), _finite_codes(rng, (N, K))
    as_, ws = np.full((rows, 4), 2.0 ** -9, np.float32), np.full((2, 4), 2.0 ** -9, np.float32)
    a, w = (torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (ac, wc))
    out = qm.fp8_matmul(a, torch.from_numpy(as_).cuda(), w, torch.from_numpy(ws).cuda(), dtype=BF16)
    want, acc = ref.matmul(ac, wc, as_, ws)
    tol = acc + ref.HALF_STEP[BF16] * (np.abs(want) + acc)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 240, 256, 272, 368, 384, 400, 496, 512, 528, 640, 656, 1008, 1024, 1040])
def test_matmul_lengths(K):
    for T, E, N in ((3, 2, 70), (90, 2, 200), (700, 2, 300)):
        _matmul_case(T, 1, E, K, N, BF16, True, K)


@pytest.mark.parametrize("N", [1, 2, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 257, 511])
def test_matmul_widths(N):
    for T, dtype in ((5, F16), (150, BF16), (600, F16)):
        _matmul_case(T, 1, 2, 272, N, dtype, False, N)


def test_matmul_nan_reaches_its_outputs_alone():
    rng = np.random.default_rng(1)
    for T in (20, 300):
        K, N = 272, 300
        ac, wc = _finite_codes(rng, (T, K)), _finite_codes(rng, (N, K))
        ac[3, 150] = 0x7f
        wc[130, 0] = 0xff
        as_, ws = np.full((T, 3), 0.01, np.float32), np.full((3, 3), 0.02, np.float32)
        as_[7, 2] = NAN
        ws[2, 1] = NAN
        a, w = (torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (ac, wc))
        out = qm.fp8_matmul(a, torch.from_numpy(as_).cuda(), w, torch.from_numpy(ws).cuda(), dtype=BF16).cpu()
        want = torch.zeros(T, N, dtype=torch.bool)
        want[3] = want[7] = True
        want[:, 130] = True
        want[:, 256:] = True
        assert torch.equal(out.isnan(), want)


def test_matmul_routes_outside_are_rows_of_zeros():
    rng = np.random.default_rng(2)
    for rows in (12, 400):
        K, N = 144, 96
        a = torch.from_numpy(_finite_codes(rng, (8, K))).cuda().view(torch.float8_e4m3fn)
        w = torch.from_numpy(_finite_codes(rng, (N, K))).cuda().view(torch.float8_e4m3fn)
        sa, sw = torch.full((8, 2), 0.125, device="cuda"), torch.full((1, 2), 0.25, device="cuda")
        order = torch.randint(0, 16, (rows,), dtype=torch.int32, device="cuda")
        order[1], order[5], order[7] = -1, 16, 2 ** 31 - 1
        out = qm.fp8_matmul(a, sa, w, sw, sorted_routes=order, top_k=2)
        assert out[[1, 5, 7]].eq(0).all()
        plain = qm.fp8_matmul(a, sa, w, sw)
        rest = (order >= 0) & (order < 16)
        # float32 sums of two blocks in either order, rounded: neighbouring values at most
        want = plain[order[rest].long() // 2]
        assert bool(((out[rest].float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs()).all())


@pytest.mark.parametrize("table", [[0, 9, 4, 20], [5, 5, 5, 5], [-7, 30, 12, 99], [20, 0, 20, 0], [3, 2, 1, 0]])
def test_matmul_bad_offsets_stay_inside(table):
    # tables that decrease or leave [0, rows] give values in out alone
    rng = np.random.default_rng(3)
    a = torch.from_numpy(_finite_codes(rng, (20, 128))).cuda().view(torch.float8_e4m3fn)
    w = torch.from_numpy(_finite_codes(rng, (3, 72, 128))).cuda().view(torch.float8_e4m3fn)
    sa, sw = torch.ones(20, 1, device="cuda"), torch.ones(3, 1, 1, device="cuda")
    pool = torch.full((22, 72), 7.0, device="cuda", dtype=BF16)
    qm.fp8_matmul(a, sa, w, sw, torch.tensor(table, dtype=torch.int32, device="cuda"), out=pool[1:21])
    assert pool[0].eq(7).all() and pool[21].eq(7).all()


def test_matmul_scales_far_apart():
    # products of scales over float32's range and sums that one block dominates
    a = torch.full((4, 256), 1.0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.full((16, 256), 1.0, device="cuda").to(torch.float8_e4m3fn)
    sa = torch.tensor([[2.0 ** 60, 2.0 ** -60], [2.0 ** -100, 2.0 ** -20], [0.0, 1.0], [-1.0, 1.0]], device="cuda")
    sw = torch.tensor([[2.0 ** -60, 2.0 ** 60]], device="cuda")
    out = qm.fp8_matmul(a, sa, w, sw)
    assert out[0].eq(256).all() and out[1].eq(128 * 2.0 ** 40).all() and out[2].eq(128 * 2.0 ** 60).all()
    assert out[3].eq(128 * 2.0 ** 60).all()


def test_matmul_two_streams_and_graph_replays():
    rng = np.random.default_rng(5)
    E, K, N, T, k = 4, 400, 200, 150, 2
    w, sw = qm.fp8_quantize_weights(torch.from_numpy(rng.normal(size=(E, N, K)).astype(np.float32)).cuda())
    sets = []
    for _ in range(2):
        ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
        _, offsets, order, _ = qm.permute(None, ids, E)
        x = torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32)).cuda()
        sets.append((x, offsets, order))

    def call(i):
        x, offsets, order = sets[i]
        return qm.fp8_matmul(*qm.fp8_quantize(x), w, sw, offsets, sorted_routes=order, top_k=k)

    want = [call(0).clone(), call(1).clone()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [None, None]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = call(i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    captured = []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            captured.append(call(i))
    for _ in range(3):
        sets[0][0].normal_()
        want[0] = call(0).clone()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_wrong_tensors():
    x = torch.randn(8, 64, device="cuda")
    (a, sa), (w, sw) = qm.fp8_quantize(x), qm.fp8_quantize_weights(x)
    for call in (lambda: qm.fp8_quantize(x.double()), lambda: qm.fp8_quantize(x.t()), lambda: qm.fp8_quantize_weights(x.t()),
                 lambda: qm.fp8_quantize_weights(x[0]), lambda: qm.fp8_dequantize(a, sa[:, :0], F32),
                 lambda: qm.fp8_dequantize(a.view(torch.uint8), sa, F32), lambda: qm.fp8_dequantize(a, sa.half(), F32),
                 lambda: qm.fp8_dequantize_weights(w, sa, F32), lambda: qm.fp8_matmul(a, sa, w, sa),
                 lambda: qm.fp8_matmul(a, sa, w[:, :32], sw), lambda: qm.fp8_matmul(a, sw, w, sw),
                 lambda: qm.fp8_matmul(a, sa, w.view(1, 1, 8, 64), sw.view(1, 1, 1, 1)),
                 lambda: qm.fp8_matmul(a, sa, w, sw, torch.zeros(3, dtype=torch.int32, device="cuda")),
                 lambda: qm.fp8_matmul(a, sa, w, sw, sorted_routes=torch.zeros(8, dtype=torch.int64, device="cuda"), top_k=1),
                 lambda: qm.fp8_matmul(a, sa, w, sw, out=x[:, :8]), lambda: qm.fp8_matmul(a, sa, w, sw, dtype=torch.float64), lambda: qm.fp8_dequantize(a, sa, torch.float64)):
        with pytest.raises(ValueError):
            call()
    pool = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    codes, scales = pool[:512].view(qm.FP8_DTYPE).view(8, 64), pool[512:544].view(F32).view(8, 1)
    with pytest.raises(ValueError, match="overlaps scales"):
        qm.fp8_dequantize(codes, scales, F32, out=pool[512:2560].view(F32).view(8, 64))
    with pytest.raises(ValueError, match="overlaps a_codes"):
        qm.fp8_matmul(codes, scales, w, sw, out=pool[256:384].view(BF16).view(8, 8))
    for call in (lambda: qm.fp8_matmul(a, sa, w, sw, dtype=F32), lambda: qm.fp8_quantize(torch.zeros(2, 24, device="cuda")), lambda: qm.fp8_quantize_weights(torch.zeros(24, 20, device="cuda")),
                 lambda: qm.fp8_quantize_weights(torch.zeros(20, 32, device="cuda"), transpose=True),
                 lambda: qm.fp8_matmul(a, sa, w, sw, sorted_routes=torch.zeros(8, dtype=torch.int32, device="cuda"), top_k=(1 << 32) + 1)):
        with pytest.raises(qm.QMoEError):
            call()
