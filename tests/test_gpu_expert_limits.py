"""GPU tests at the largest sizes that the sort by expert and back and the MXFP4 operators admit."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _small_values(g, rows, K):
    """MXFP4 operands of 0, 0.5 and 1 with scale 1: sums of up to 2^20 products are exact in float32."""
    low = torch.randint(0, 3, (2, rows, K // 2), generator=g, device="cuda")
    sign = torch.randint(0, 2, (2, rows, K // 2), generator=g, device="cuda") * 8
    code = (low | sign).to(torch.uint8)
    return code[0] | (code[1] << 4), torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("K", [1 << 20, (1 << 20) - 32, (1 << 20) - 512])
def test_matmul_longest_rows(K):
    g = torch.Generator(device="cuda").manual_seed(K)
    a, w = _small_values(g, 3, K), _small_values(g, 70, K)
    want = qm.mx_dequantize(*a, F32).double() @ qm.mx_dequantize(*w, F32).double().T.contiguous()
    assert torch.equal(qm.mx_matmul(*a, *w, dtype=F32).double(), want)


def test_matmul_most_rows():
    g = torch.Generator(device="cuda").manual_seed(0)
    rows, K, N = (1 << 24) - 1, 32, 3
    a, w = _small_values(g, rows, K), _small_values(g, 2 * N, K)
    w = [t.view(2, N, -1) for t in w]
    cut = 1 << 23
    off = torch.tensor([0, cut + 77, rows - 5], dtype=torch.int32, device="cuda")
    out = qm.mx_matmul(*a, *w, off, dtype=F32)
    assert out[rows - 5:].eq(0).all()
    wv = qm.mx_dequantize(*w, F32).double()
    for lo, hi, e in ((0, 300, 0), (cut - 200, cut + 77, 0), (cut + 77, cut + 400, 1), (rows - 300, rows - 5, 1)):
        av = qm.mx_dequantize(a[0][lo:hi].contiguous(), a[1][lo:hi].contiguous(), F32).double()
        assert torch.equal(out[lo:hi].double(), av @ wv[e].T.contiguous())


def test_matmul_most_rows_behind_routes():
    # codes of just under 2^31 bytes; routes to the last rows, to one row often and past the end
    g = torch.Generator(device="cuda").manual_seed(1)
    K, N = 4096, 40
    A = ((1 << 31) - 1) // (K // 2)
    codes = torch.zeros((A, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((A, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-50:] = _small_values(g, 50, K)[0]
    w = _small_values(g, N, K)
    named = torch.tensor([A - 1, 0, A - 50, A, A - 2, A - 1, -1, 2 ** 31 - 1] * 30, dtype=torch.int32, device="cuda")
    out = qm.mx_matmul(codes, scales, *w, sorted_routes=named, top_k=1, dtype=F32).double()
    wv = qm.mx_dequantize(*w, F32).double().T.contiguous()
    last = qm.mx_dequantize(codes[-50:].contiguous(), scales[-50:].contiguous(), F32).double() @ wv
    want = torch.zeros_like(out)
    for at, row in ((0, 49), (2, 0), (4, 48), (5, 49)):
        want[at::8] = last[row]
    assert torch.equal(out, want)
    with pytest.raises(qm.QMoEError):
        qm.mx_matmul(torch.empty((A + 1, K // 2), dtype=torch.uint8, device="cuda"),
                     torch.empty((A + 1, K // 32), dtype=torch.uint8, device="cuda"), *w, sorted_routes=named, top_k=1)


def test_matmul_most_experts():
    g = torch.Generator(device="cuda").manual_seed(2)
    E, N, K = 1024, 17, 1056
    counts = torch.randint(0, 3, (E,), generator=g, device="cuda")
    off = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int()
    rows = int(off[-1])
    a, w = _small_values(g, rows, K), _small_values(g, E * N, K)
    w = [t.view(E, N, -1) for t in w]
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    av, wv = qm.mx_dequantize(*a, F32).double(), qm.mx_dequantize(*w, F32).double()
    want = (av[:, None] * wv[expert]).sum(-1)
    assert torch.equal(qm.mx_matmul(*a, *w, off, dtype=F32).double(), want)


@pytest.mark.parametrize("top_k,E", [(1, 1024), (256, 5)])
def test_permute_most_tokens(top_k, E):
    # route r goes to expert r % (E + 1), the last of which drops it: every map is known
    T = (1 << 23) - 1
    R = T * top_k
    ids = torch.arange(R, dtype=torch.int32, device="cuda")
    ids.remainder_(E + 1)
    rows, offsets, order, rr = qm.permute(None, ids.view(T, top_k), E)
    del ids
    assert rows is None
    count = [(R - e + E) // (E + 1) for e in range(E + 1)]
    start = [sum(count[:e]) for e in range(E + 1)]
    assert offsets.tolist() == start
    for e in range(E + 1):
        seg = order[start[e]:start[e] + count[e]]
        assert int(seg[0]) == e and int(seg[-1]) == e + (count[e] - 1) * (E + 1)
        if count[e] > 1:
            assert bool((seg[1:] - seg[:-1] == E + 1).all())
        if e < 6 or e == E:
            mine = rr.view(-1)[e::E + 1]
            at = torch.arange(start[e], start[e] + count[e], dtype=torch.int32, device="cuda")
            assert torch.equal(mine, at if e < E else -1 - at)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_widest_rows(dtype):
    T, k, H, E = 3, 2, 1 << 20, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    ids = torch.tensor([[1, 3], [-1, 0], [2, 1]], dtype=torch.int32, device="cuda")
    rows, offsets, order, rr = qm.permute(x, ids, E)
    want = x[order.long() // k]
    want[5] = 0
    assert torch.equal(rows, want)
    w = torch.tensor([[0.75, 0.25], [9.0, 1.0], [0.5, 0.5]], device="cuda")
    # 0.75 x + 0.25 x and 0.5 x + 0.5 x: the sum of two float32 products, at most one step of float32 from x
    got = qm.unpermute(rows, rr, w).double()
    assert bool(((got - x.double()).abs() <= (2 * ref.U32 + ref.HALF_STEP[dtype]) * x.double().abs()).all())
    gr, gw = qm.unpermute_backward(x, rows, rr, w)
    dots = (x.double()[:, None] * rows.double()[torch.where(rr >= 0, rr, 0).long()]) * (rr >= 0)[..., None]
    assert bool(((gw.double() - dots.sum(-1)).abs() <= (H + 1) * ref.U32 * dots.abs().sum(-1)).all())
    assert gr[5].eq(0).all() and torch.equal(gr[int(rr[2, 0])], (x[2].float() * 0.5).to(dtype))


def test_quantize_past_32_bits():
    # 8.6 billion values: the indexes of values, codes and groups of eight pass 2^32, 2^31 and 2^30
    rows, K = (1 << 19) + 1, 1 << 14
    x = torch.zeros((rows, K), dtype=F16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    x[-1] = torch.randn(K, generator=g, device="cuda").to(F16)
    codes, scales = qm.mx_quantize(x)
    last = qm.mx_quantize(x[-1].clone())
    assert torch.equal(codes[-1], last[0]) and torch.equal(scales[-1], last[1])
    assert codes[rows // 2].eq(0).all() and codes[-2].eq(0).all() and scales[-2].eq(0).all()
    del x
    back = qm.mx_dequantize(codes, scales, F16)
    assert torch.equal(back[-1], qm.mx_dequantize(*last, F16)) and back[-2].eq(0).all()


def test_quantize_columns_of_most_matrices():
    E = 65535
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(E, 32, 3, generator=g, device="cuda").to(BF16)
    codes, scales = qm.mx_quantize(x, transpose=True)
    want = qm.mx_quantize(x.transpose(1, 2).contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    with pytest.raises(qm.QMoEError):
        qm.mx_quantize(torch.zeros(E + 1, 32, 1, device="cuda"), transpose=True)
