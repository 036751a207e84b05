"""Refusals of the sort by expert and back and of the MXFP4 operators, without a GPU: every invalid
argument is rejected before the device is touched, and the binding checks its tensors."""
from __future__ import annotations

import os
import re

import pytest
import torch

import quantized_mixture_experts_route_amd as qm

FAKE = 1 << 20  # a non-NULL address; never dereferenced on these paths
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "qmoe.h")).read()
    assert re.search(r"#define QMOE_DTYPE_F32 (\d+)", text).group(1) == str(qm.DTYPE_F32)


def test_permute_workspace_size():
    size = qm.permute_workspace_size
    assert size(8, 2, 8) == 0 and size(0, 2, 8) == 0  # one launch, no workspace
    assert size(100000, 8, 64) > 0 and size(100000, 8, 64) % 4 == 0
    assert size(100000, 8, 1024) > size(100000, 8, 64)
    for bad in ((-1, 2, 8), (8, 0, 8), (8, 1025, 8), (8, 2, 0), (8, 2, 1025), (1 << 23, 2, 8), (1 << 22, 1024, 8)):
        assert size(*bad) == 0
    for T in (1 << 14, 1 << 17, 1 << 20, (1 << 23) - 1):  # at most a span's counters per 1024 routes
        assert size(T, 2, 8) <= (2 * T // 1024 + 3) * 9 * 4


def _call(name, defaults, kw):
    args = dict(defaults, **kw)
    rc = getattr(qm.load_library(), name)(*args.values())
    return rc


PERMUTE = dict(hidden=FAKE, stride=64, T=4, H=64, dtype=1, ids=FAKE, k=2, E=8, rows=FAKE, offsets=FAKE,
               order=FAKE, route_rows=FAKE, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), qm.ERR_INVALID_ARG), (dict(T=1 << 23), qm.ERR_UNSUPPORTED),
    (dict(k=0), qm.ERR_INVALID_ARG), (dict(k=1025), qm.ERR_INVALID_ARG),
    (dict(T=1 << 22, k=512), qm.ERR_INVALID_ARG),
    (dict(E=0), qm.ERR_INVALID_ARG), (dict(E=1025), qm.ERR_INVALID_ARG),
    (dict(H=0), qm.ERR_INVALID_ARG), (dict(H=(1 << 20) + 1, stride=1 << 21), qm.ERR_UNSUPPORTED),
    (dict(dtype=0), qm.ERR_INVALID_ARG), (dict(dtype=4), qm.ERR_INVALID_ARG),
    (dict(stride=63), qm.ERR_INVALID_ARG), (dict(stride=-64), qm.ERR_INVALID_ARG),
    (dict(stride=1 << 62), qm.ERR_INVALID_ARG),
    (dict(hidden=None), qm.ERR_INVALID_ARG), (dict(rows=None), qm.ERR_INVALID_ARG),
    (dict(hidden=FAKE + 1), qm.ERR_INVALID_ARG), (dict(dtype=3, rows=FAKE + 2), qm.ERR_INVALID_ARG),
    (dict(ids=None), qm.ERR_INVALID_ARG), (dict(offsets=None), qm.ERR_INVALID_ARG),
    (dict(order=None), qm.ERR_INVALID_ARG), (dict(route_rows=None), qm.ERR_INVALID_ARG),
    (dict(route_rows=FAKE + 2), qm.ERR_INVALID_ARG),
    (dict(T=100000), qm.ERR_WORKSPACE), (dict(T=100000, ws=FAKE, ws_bytes=64), qm.ERR_WORKSPACE),
    (dict(T=100000, ws_bytes=1 << 30), qm.ERR_INVALID_ARG),
    (dict(T=0, offsets=None), qm.ERR_INVALID_ARG),
])
def test_permute_refuses(kw, code):
    assert _call("qmoe_permute", PERMUTE, kw) == code, qm.last_error()
    assert qm.last_error().startswith("qmoe: ")


BACK = dict(rows=FAKE, stride=64, route_rows=FAKE, weights=FAKE, T=4, k=2, H=64, dtype=2, out=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), qm.ERR_INVALID_ARG), (dict(T=1 << 23), qm.ERR_UNSUPPORTED), (dict(k=0), qm.ERR_INVALID_ARG),
    (dict(H=0), qm.ERR_INVALID_ARG), (dict(H=1 << 21, stride=1 << 21), qm.ERR_UNSUPPORTED),
    (dict(dtype=5), qm.ERR_INVALID_ARG), (dict(stride=8), qm.ERR_INVALID_ARG),
    (dict(rows=None), qm.ERR_INVALID_ARG), (dict(route_rows=None), qm.ERR_INVALID_ARG),
    (dict(weights=FAKE + 1), qm.ERR_INVALID_ARG), (dict(out=None), qm.ERR_INVALID_ARG),
    (dict(out=FAKE + 1), qm.ERR_INVALID_ARG),
])
def test_unpermute_refuses(kw, code):
    assert _call("qmoe_unpermute", BACK, kw) == code, qm.last_error()


GRAD = dict(grad=FAKE, gstride=64, rows=FAKE, stride=64, route_rows=FAKE, weights=None, T=4, k=2, H=64,
            dtype=3, grad_rows=FAKE, grad_weights=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), qm.ERR_INVALID_ARG), (dict(k=1025), qm.ERR_INVALID_ARG), (dict(H=-1), qm.ERR_INVALID_ARG),
    (dict(dtype=0), qm.ERR_INVALID_ARG), (dict(gstride=63), qm.ERR_INVALID_ARG),
    (dict(stride=63), qm.ERR_INVALID_ARG), (dict(grad=None), qm.ERR_INVALID_ARG),
    (dict(rows=None), qm.ERR_INVALID_ARG), (dict(grad_weights=None), qm.ERR_INVALID_ARG),
    (dict(grad_rows=None), qm.ERR_INVALID_ARG), (dict(grad_rows=FAKE + 2), qm.ERR_INVALID_ARG),
    (dict(route_rows=None), qm.ERR_INVALID_ARG),
])
def test_unpermute_backward_refuses(kw, code):
    assert _call("qmoe_unpermute_backward", GRAD, kw) == code, qm.last_error()


QUANT = dict(x=FAKE, stride=64, rows=4, K=64, dtype=2, codes=FAKE, scales=FAKE, stream=None)
COLUMNS = dict(x=FAKE, E=2, rows=64, K=7, dtype=2, codes=FAKE, scales=FAKE, stream=None)
DEQUANT = dict(codes=FAKE, scales=FAKE, rows=4, K=64, dtype=2, out=FAKE, stream=None)


@pytest.mark.parametrize("name,defaults,kw,code", [
    ("qmoe_mx_quantize", QUANT, dict(rows=-1), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(K=0), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(K=48), qm.ERR_UNSUPPORTED),
    ("qmoe_mx_quantize", QUANT, dict(rows=1 << 40), qm.ERR_UNSUPPORTED),
    ("qmoe_mx_quantize", QUANT, dict(dtype=0), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(stride=32), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(x=None), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(codes=FAKE + 8), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize", QUANT, dict(scales=None), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(E=-1), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(rows=0), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(rows=40), qm.ERR_UNSUPPORTED),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(E=1 << 16), qm.ERR_UNSUPPORTED),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(x=None), qm.ERR_INVALID_ARG),
    ("qmoe_mx_quantize_columns", COLUMNS, dict(codes=None), qm.ERR_INVALID_ARG),
    ("qmoe_mx_dequantize", DEQUANT, dict(rows=-2), qm.ERR_INVALID_ARG),
    ("qmoe_mx_dequantize", DEQUANT, dict(K=33), qm.ERR_UNSUPPORTED),
    ("qmoe_mx_dequantize", DEQUANT, dict(dtype=7), qm.ERR_INVALID_ARG),
    ("qmoe_mx_dequantize", DEQUANT, dict(out=FAKE + 1), qm.ERR_INVALID_ARG),
    ("qmoe_mx_dequantize", DEQUANT, dict(scales=None), qm.ERR_INVALID_ARG),
])
def test_conversions_refuse(name, defaults, kw, code):
    assert _call(name, defaults, kw) == code, qm.last_error()


MATMUL = dict(a=FAKE, sa=FAKE, a_rows=8, w=FAKE, sw=FAKE, E=4, N=64, K=64, offsets=FAKE, order=None, k=1,
              rows=8, dtype=2, out=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), qm.ERR_INVALID_ARG), (dict(E=1025), qm.ERR_INVALID_ARG), (dict(N=0), qm.ERR_INVALID_ARG),
    (dict(K=0), qm.ERR_INVALID_ARG), (dict(K=80), qm.ERR_UNSUPPORTED), (dict(K=(1 << 20) + 32), qm.ERR_UNSUPPORTED),
    (dict(N=1 << 21), qm.ERR_UNSUPPORTED), (dict(rows=-1), qm.ERR_INVALID_ARG),
    (dict(rows=1 << 24, a_rows=1 << 24), qm.ERR_UNSUPPORTED), (dict(rows=9), qm.ERR_INVALID_ARG),
    (dict(a_rows=-1), qm.ERR_INVALID_ARG), (dict(a_rows=0, order=FAKE), qm.ERR_INVALID_ARG),
    (dict(dtype=0), qm.ERR_INVALID_ARG), (dict(k=0), qm.ERR_INVALID_ARG), (dict(offsets=None), qm.ERR_INVALID_ARG),
    (dict(a=None), qm.ERR_INVALID_ARG), (dict(a=FAKE + 4), qm.ERR_INVALID_ARG), (dict(sa=None), qm.ERR_INVALID_ARG),
    (dict(w=FAKE + 8), qm.ERR_INVALID_ARG), (dict(sw=None), qm.ERR_INVALID_ARG),
    (dict(offsets=FAKE + 1), qm.ERR_INVALID_ARG), (dict(order=FAKE + 2), qm.ERR_INVALID_ARG),
    (dict(out=None), qm.ERR_INVALID_ARG), (dict(dtype=3, out=FAKE + 2), qm.ERR_INVALID_ARG),
])
def test_matmul_refuses(kw, code):
    assert _call("qmoe_mx_matmul", MATMUL, kw) == code, qm.last_error()


def test_empty_calls_touch_nothing():
    for name, defaults, kw in (("qmoe_unpermute", BACK, dict(T=0, rows=None, out=None, route_rows=None)),
                               ("qmoe_unpermute_backward", GRAD, dict(T=0, grad=None)),
                               ("qmoe_mx_quantize", QUANT, dict(rows=0, x=None)),
                               ("qmoe_mx_quantize_columns", COLUMNS, dict(E=0, x=None)),
                               ("qmoe_mx_dequantize", DEQUANT, dict(rows=0, out=None)),
                               ("qmoe_mx_matmul", MATMUL, dict(rows=0, a_rows=0, out=None))):
        assert _call(name, defaults, kw) == qm.OK, (name, qm.last_error())
        assert qm.last_error() == ""


def test_binding_refuses_cpu_tensors_and_shapes():
    ids = torch.zeros((4, 2), dtype=torch.int32)
    x = torch.zeros((4, 64))
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    for call in (lambda: qm.permute(x, ids, 4), lambda: qm.permute(x, ids[0], 4), lambda: qm.permute(x, None, 4),
                 lambda: qm.unpermute(x, ids), lambda: qm.unpermute(x, ids.reshape(-1)),
                 lambda: qm.unpermute_backward(x, x, ids), lambda: qm.mx_quantize(x),
                 lambda: qm.mx_quantize(x, transpose=True), lambda: qm.mx_dequantize(codes, scales, torch.float16),
                 lambda: qm.mx_dequantize(codes, scales, torch.float64),
                 lambda: qm.mx_matmul(codes, scales, codes, scales)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_device():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 64), device="cuda")
    rows = torch.zeros((8, 64), device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    codes = torch.zeros((4, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    for call in (lambda: qm.permute(x.double(), ids, 4), lambda: qm.permute(x[:3], ids, 4),
                 lambda: qm.permute(x, ids.long(), 4), lambda: qm.permute(x.t(), ids, 4),
                 lambda: qm.permute(x[:1].expand(4, 64), ids, 4), lambda: qm.permute(x, ids[:, :1], 4),
                 lambda: qm.unpermute(x, ids), lambda: qm.unpermute(rows, ids, w.half()),
                 lambda: qm.unpermute(rows, ids, w, out=x.half()), lambda: qm.unpermute(rows, ids, w.cpu()),
                 lambda: qm.unpermute_backward(x, rows.half(), ids, w),
                 lambda: qm.unpermute_backward(x[:2], rows, ids, w), lambda: qm.mx_quantize(x.int()),
                 lambda: qm.mx_quantize(x.t(), transpose=True), lambda: qm.mx_quantize(x[0, 0]),
                 lambda: qm.mx_dequantize(codes, scales[:, :1], torch.float16),
                 lambda: qm.mx_dequantize(codes, scales[:3], torch.float16),
                 lambda: qm.mx_matmul(codes, scales, codes[:, :16], scales[:, :1]),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, ids),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, out=w),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, sorted_routes=ids),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, dtype=torch.int8)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.permute(x, ids, 0), lambda: qm.permute(x, ids, 1025), lambda: qm.permute(x, ids[:, :0], 4),
                 lambda: qm.mx_quantize(x[:, :40]), lambda: qm.mx_quantize(x, transpose=True),
                 lambda: qm.mx_matmul(codes, scales, codes[None].repeat(2, 1, 1), scales[None].repeat(2, 1, 1)),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, top_k=0),
                 lambda: qm.permute(None, torch.zeros((100000, 2), dtype=torch.int32, device="cuda"), 8,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(qm.QMoEError):
            call()
