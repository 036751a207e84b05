"""GPU tests at the largest sizes that routing by scores, the 8-bit operators and the gated activation admit, and
of sizes that do not fit the 32 bits in which the library takes them."""
from __future__ import annotations

import math

import pytest
import torch

import quantized_mixture_experts_route_amd as qm

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
WIDE = 1 << 32


def _codes(g, *shape):
    """Codes of 0, 0.5, 1 and -1, in bytes: sums of up to 2^20 of their products are exact in float32."""
    named = torch.tensor([0x00, 0x30, 0x38, 0xb8], dtype=torch.uint8, device="cuda")
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for row in out.view(-1, shape[-1]).split(max((1 << 28) // shape[-1], 1)):
        row.copy_(named[torch.randint(0, 4, row.shape, generator=g, device="cuda", dtype=torch.uint8).long()])
    return out.view(qm.FP8_DTYPE)


def _ones(*shape):
    return torch.ones(shape, dtype=F32, device="cuda")


def _blocks(n):
    return -(-n // 128)


def _scales(codes):
    return _ones(*codes.shape[:-1], _blocks(codes.shape[-1]))


def _squares(w):
    return _ones(*w.shape[:-2], _blocks(w.shape[-2]), _blocks(w.shape[-1]))


def _product(a, w):
    """Exact, for codes with scales of 1."""
    a, w = (qm.fp8_dequantize(t.contiguous(), _scales(t), F32).double() for t in (a, w))
    return a @ w.T.contiguous()


@pytest.mark.parametrize("rows,N", [(3, 70), (300, 520)])
@pytest.mark.parametrize("K", [1 << 20, (1 << 20) - 16])
def test_matmul_longest_rows(rows, N, K):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    a, w = _codes(g, rows, K), _codes(g, N, K)
    out = qm.fp8_matmul(a, _scales(a), w, _squares(w), dtype=BF16)
    assert torch.equal(out, _product(a, w).to(BF16))


@pytest.mark.parametrize("rows,N", [((1 << 24) - 1, 3), ((1 << 23) + 5, 300)])  # the second: results behind 4 GiB
def test_matmul_most_rows(rows, N):
    g = torch.Generator(device="cuda").manual_seed(N)
    a, w = _codes(g, rows, 16), _codes(g, 2, N, 16)
    cut = rows // 2 + 77
    off = torch.tensor([0, cut, rows - 5], dtype=torch.int32, device="cuda")
    out = qm.fp8_matmul(a, _scales(a), w, _squares(w), off, dtype=F16)
    assert out[rows - 5:].eq(0).all()
    for lo, hi, e in ((0, 300, 0), (cut - 300, cut, 0), (cut, cut + 300, 1), (rows - 300, rows - 5, 1)):
        assert torch.equal(out[lo:hi], _product(a[lo:hi], w[e]).to(F16))


def test_matmul_most_rows_behind_routes():
    # codes of just under 2^31 bytes; routes to the last rows, to one row often and past the end
    g = torch.Generator(device="cuda").manual_seed(1)
    K, N = 2048, 40
    A = ((1 << 31) - 1) // K
    codes = torch.zeros((A, K), dtype=torch.uint8, device="cuda")
    codes[-50:] = _codes(g, 50, K).view(torch.uint8)
    codes = codes.view(qm.FP8_DTYPE)
    w = _codes(g, N, K)
    named = [A - 1, 0, A - 50, A, A - 2, A - 1, -1, 2 ** 31 - 1]
    for repeats in (2, 3000):  # few rows and tiles
        routes = torch.tensor(named * repeats, dtype=torch.int32, device="cuda")
        out = qm.fp8_matmul(codes, _scales(codes), w, _squares(w), sorted_routes=routes, top_k=1, dtype=BF16)
        last = _product(codes[-50:], w).to(BF16)
        want = torch.zeros_like(out)
        for at, row in ((0, 49), (2, 0), (4, 48), (5, 49)):
            want[at::8] = last[row]
        assert torch.equal(out, want)
    more = torch.empty((A + 1, K), dtype=torch.uint8, device="cuda").view(qm.FP8_DTYPE)
    with pytest.raises(qm.QMoEError) as e:
        qm.fp8_matmul(more, _scales(more), w, _squares(w), sorted_routes=routes, top_k=1)
    assert e.value.code == qm.ERR_UNSUPPORTED


@pytest.mark.parametrize("rows", [30, 2000])
def test_matmul_weights_behind_4_gib(rows):
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K = 32784, 65536
    w = _codes(g, 3, N, K)
    a = _codes(g, rows, K)
    off = torch.tensor([0, 4, 6, rows], dtype=torch.int32, device="cuda")
    out = qm.fp8_matmul(a, _scales(a), w, _squares(w), off, dtype=BF16)
    for lo, hi, e in ((0, 4, 0), (4, 6, 1), (6, rows, 2)):
        for n in (slice(0, 200), slice(N - 200, N)):
            assert torch.equal(out[lo:hi, n], _product(a[lo:hi], w[e, n]).to(BF16))


def test_matmul_rows_behind_4_gib():
    g = torch.Generator(device="cuda").manual_seed(4)
    rows, N, K = 70000, 40, 65536
    a, w = _codes(g, rows, K), _codes(g, N, K)
    out = qm.fp8_matmul(a, _scales(a), w, _squares(w), dtype=F16)
    for lo, hi in ((0, 100), (rows // 2, rows // 2 + 100), (rows - 100, rows)):
        assert torch.equal(out[lo:hi], _product(a[lo:hi], w).to(F16))


def test_matmul_most_experts():
    g = torch.Generator(device="cuda").manual_seed(5)
    E, N, K, rows = 1024, 17, 1040, 3000
    a, w = _codes(g, rows, K), _codes(g, E, N, K)
    counts = torch.bincount(torch.randint(0, E, (rows - 9,), generator=g, device="cuda"), minlength=E)
    off = torch.cat((torch.zeros(1, device="cuda"), counts.cumsum(0))).int()
    out = qm.fp8_matmul(a, _scales(a), w, _squares(w), off, dtype=F16)
    av, wv = (qm.fp8_dequantize(t, _scales(t), F32).double() for t in (a, w))
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    want = (av[:rows - 9, None] * wv[expert]).sum(2)
    assert torch.equal(out[:rows - 9], want.to(F16)) and out[rows - 9:].eq(0).all()


def test_conversions_of_more_values_than_threads():
    rows, K = (1 << 27) + 3, 16  # 16 threads a row: above 2^31
    x = torch.empty((rows, K), dtype=F16, device="cuda").normal_()
    codes, scales = qm.fp8_quantize(x)
    back = qm.fp8_dequantize(codes, scales, F16)
    for lo, hi in ((0, 500), (rows // 2, rows // 2 + 500), (rows - 500, rows)):
        c, s = qm.fp8_quantize(x[lo:hi])
        assert torch.equal(codes[lo:hi].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[lo:hi], s)
        assert torch.equal(back[lo:hi], qm.fp8_dequantize(c, s, F16))


def test_conversions_of_the_longest_rows():
    K = 1 << 20
    x = torch.empty((130, K), dtype=BF16, device="cuda").normal_()
    codes, scales = qm.fp8_quantize(x)
    squares = qm.fp8_quantize_weights(x)
    turned = qm.fp8_quantize_weights(x.T.contiguous(), transpose=True)  # 2^20 rows
    assert torch.equal(squares[0].view(torch.uint8), turned[0].view(torch.uint8)) and torch.equal(squares[1], turned[1])
    back, back_squares = qm.fp8_dequantize(codes, scales, BF16), qm.fp8_dequantize_weights(*squares, BF16)
    for lo in (0, K // 2, K - 1024):
        part = x[:, lo:lo + 1024]
        c, s = qm.fp8_quantize(part)
        assert torch.equal(codes[:, lo:lo + 1024].view(torch.uint8), c.view(torch.uint8))
        assert torch.equal(back[:, lo:lo + 1024], qm.fp8_dequantize(c, s, BF16))
        c, s = qm.fp8_quantize_weights(part.contiguous())
        assert torch.equal(squares[0][:, lo:lo + 1024].view(torch.uint8), c.view(torch.uint8))
        assert torch.equal(back_squares[:, lo:lo + 1024], qm.fp8_dequantize_weights(c, s, BF16))


def test_conversions_of_the_most_matrices():
    x = torch.empty((65535, 3, 16), dtype=F32, device="cuda").normal_()
    codes, scales = qm.fp8_quantize_weights(x)
    c, s = qm.fp8_quantize_weights(x[-7:])
    assert torch.equal(codes[-7:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-7:], s)
    back = qm.fp8_dequantize_weights(codes, scales, F32)
    assert bool(((back - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, scales.view(-1, 1, 1) * 2.0 ** -10)).all())


@pytest.mark.parametrize("rows,I", [((1 << 31) + 5, 1), (3, 1 << 19), ((1 << 18) + 3, 16384)])
@pytest.mark.parametrize("layout", [qm.SWIGLU_INTERLEAVED, qm.SWIGLU_HALVES])
def test_activation_of_the_most_values(rows, I, layout):
    y = torch.empty((rows, 2 * I), dtype=F16, device="cuda").normal_()
    out, grad = qm.activate(y, swiglu_fusion=layout), qm.activate_backward(y[:, :I], y, swiglu_fusion=layout)
    eight = qm.activate_fp8(y, swiglu_fusion=layout) if I % 16 == 0 else None
    n = min(rows, 100)
    for lo in (0, (rows - n) // 2, rows - n):
        part = y[lo:lo + n].clone()
        if layout == qm.SWIGLU_INTERLEAVED:
            part = torch.cat((part[:, ::2], part[:, 1::2]), 1)
        # in the other layout, and by columns where the row is long
        for j in range(0, I, 16384):
            w = min(16384, I - j)
            at = torch.stack((part[:, j:j + w], part[:, I + j:I + j + w]), 2).flatten(1)
            assert torch.equal(out[lo:lo + n, j:j + w], qm.activate(at))
            d = qm.activate_backward(y[lo:lo + n, j:j + w].contiguous(), at)
            to = grad[lo:lo + n]
            gate, up = (to[:, ::2], to[:, 1::2]) if layout == qm.SWIGLU_INTERLEAVED else (to[:, :I], to[:, I:])
            assert torch.equal(gate[:, j:j + w], d[:, ::2]) and torch.equal(up[:, j:j + w], d[:, 1::2])
            if eight is not None:
                c, s = qm.activate_fp8(at)
                assert torch.equal(eight[0][lo:lo + n, j:j + w].view(torch.uint8), c.view(torch.uint8))
                assert torch.equal(eight[1][lo:lo + n, j // 128:j // 128 + s.shape[1]], s)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
def test_routes_of_the_most_tokens(score):
    T, E = (1 << 23) - 1, 64
    logits = torch.empty((T, 300), dtype=F16, device="cuda").normal_()[:, 100:100 + E]  # 5 GB apart
    ids, w = qm.route_scores(logits, 6, score=score, n_groups=8, top_groups=3, group_top=2)
    grad = qm.route_scores_backward(w, logits, ids, score=score)
    for lo in (0, T // 2, T - 300):
        part = logits[lo:lo + 300].contiguous()
        i, v = qm.route_scores(part, 6, score=score, n_groups=8, top_groups=3, group_top=2)
        assert torch.equal(ids[lo:lo + 300], i) and torch.equal(w[lo:lo + 300], v)
        assert torch.equal(grad[lo:lo + 300], qm.route_scores_backward(v, part, i, score=score))


def test_calls_refuse_wide_sizes():
    x = torch.zeros((4, 64), device="cuda")
    ids, w = qm.route_scores(x, 2)
    codes, scales = qm.fp8_quantize(x)
    order = torch.arange(4, dtype=torch.int32, device="cuda")
    wide = torch.empty(WIDE + 32, dtype=F16, device="cuda").view(1, -1)
    wide_codes = torch.empty(WIDE + 16, dtype=torch.uint8, device="cuda").view(1, -1).view(qm.FP8_DTYPE)
    wide_scales = torch.empty((1, math.ceil((WIDE + 16) / 128)), device="cuda")
    one = torch.ones((1, 1), device="cuda")
    calls = [lambda: qm.route_scores(wide, 2), lambda: qm.route_scores_backward(one, wide, one.int()),
             lambda: qm.fp8_quantize(wide), lambda: qm.fp8_quantize(wide[0]), lambda: qm.fp8_quantize_weights(wide),
             lambda: qm.fp8_quantize_weights(wide.T.contiguous(), transpose=True),
             lambda: qm.fp8_dequantize(wide_codes, wide_scales, F16),
             lambda: qm.fp8_dequantize_weights(wide_codes, wide_scales, F16),
             lambda: qm.fp8_matmul(wide_codes, wide_scales, wide_codes, wide_scales),
             lambda: qm.fp8_matmul(codes, scales, codes, scales[:1], sorted_routes=order, top_k=WIDE + 1),
             lambda: qm.activate(wide), lambda: qm.activate_fp8(wide), lambda: qm.activate_backward(wide, wide)]
    for kw in (dict(top_k=WIDE + 2), dict(score=WIDE), dict(n_groups=WIDE + 1), dict(top_groups=WIDE + 1), dict(group_top=WIDE + 1)):
        calls.append(lambda kw=kw: qm.route_scores(x, **{"top_k": 2, **kw}))
    calls.append(lambda: qm.route_scores_backward(w, x, ids, score=WIDE + 1))
    for call in (qm.activate, qm.activate_fp8, lambda y, **kw: qm.activate_backward(y[:, :32], y, **kw)):
        calls += [lambda call=call: call(x, activation=WIDE), lambda call=call: call(x, swiglu_fusion=WIDE + 1)]
    for i, call in enumerate(calls):
        with pytest.raises(qm.QMoEError) as e:
            call()
        assert e.value.code == qm.ERR_UNSUPPORTED, i
