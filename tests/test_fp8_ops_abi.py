"""Refusals of routing by scores, the 8-bit floating point operators and the gated activation, without a GPU:
every invalid argument is rejected before the device is touched, and the binding checks its tensors."""
from __future__ import annotations

import os
import re

import pytest
import torch

import quantized_mixture_experts_route_amd as qm

FAKE = 1 << 20  # a non-NULL address; never dereferenced on these paths
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP = qm.ERR_INVALID_ARG, qm.ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def _call(name, defaults, kw):
    assert set(kw) <= set(defaults), kw
    return getattr(qm.load_library(), name)(*dict(defaults, **kw).values())


def _refused(name, defaults, kw, code):
    assert _call(name, defaults, kw) == code, qm.last_error()
    assert qm.last_error().startswith("qmoe: ")


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "qmoe.h")).read()
    for name in ("SCORE_SOFTMAX", "SCORE_SIGMOID", "SWIGLU_INTERLEAVED", "SWIGLU_HALVES"):
        assert re.search(rf"#define QMOE_{name} (\d+)", text).group(1) == str(getattr(qm, name))


ROUTE = dict(logits=FAKE, stride=64, T=4, E=64, dtype=3, bias=FAKE, k=4, score=1, groups=8, kept=4, best=2, norm=1,
             scale=1.0, ids=FAKE, weights=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(T=1 << 23), UNSUP), (dict(E=0), BAD), (dict(E=1025, stride=1025), BAD),
    (dict(dtype=0), BAD), (dict(dtype=4), BAD), (dict(k=0), BAD), (dict(k=65, E=512, stride=512), UNSUP),
    (dict(k=65), BAD), (dict(k=33), BAD), (dict(score=2), BAD), (dict(score=-1), BAD),
    (dict(groups=0), BAD), (dict(groups=7), BAD), (dict(groups=128, E=128, stride=128, kept=128), UNSUP),
    (dict(kept=0), BAD), (dict(kept=9), BAD), (dict(best=0), BAD), (dict(best=3), BAD),
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(stride=63), BAD), (dict(stride=-1), BAD),
    (dict(stride=1 << 62), BAD), (dict(logits=None), BAD), (dict(logits=FAKE + 2), BAD), (dict(logits=FAKE + 1, dtype=1), BAD),
    (dict(bias=FAKE + 2), BAD), (dict(ids=None), BAD), (dict(ids=FAKE + 1), BAD), (dict(weights=None), BAD),
])
def test_route_scores_refuses(kw, code):
    _refused("qmoe_route_scores", ROUTE, kw, code)


ROUTE_GRAD = dict(grad=FAKE, logits=FAKE, stride=64, ids=FAKE, T=4, E=64, dtype=2, k=4, score=0, norm=0, scale=1.0,
                  out=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(T=1 << 23), UNSUP), (dict(E=0), BAD), (dict(k=0), BAD), (dict(k=65), BAD), (dict(dtype=9), BAD),
    (dict(score=5), BAD), (dict(scale=-INF), BAD), (dict(stride=1), BAD), (dict(grad=None), BAD),
    (dict(grad=FAKE + 2), BAD), (dict(logits=None), BAD), (dict(ids=None), BAD), (dict(out=None), BAD), (dict(out=FAKE + 1), BAD),
])
def test_route_scores_backward_refuses(kw, code):
    _refused("qmoe_route_scores_backward", ROUTE_GRAD, kw, code)


QUANT = dict(x=FAKE, stride=64, rows=4, K=64, dtype=1, codes=FAKE, scales=FAKE, stream=None)
SQUARES = dict(x=FAKE, E=2, rows=64, K=64, dtype=1, transpose=0, codes=FAKE, scales=FAKE, stream=None)
BACK = dict(codes=FAKE, scales=FAKE, rows=4, K=64, dtype=1, out=FAKE, stream=None)
BACK_SQUARES = dict(codes=FAKE, scales=FAKE, E=2, rows=4, K=64, dtype=1, out=FAKE, stream=None)


@pytest.mark.parametrize("name,defaults,kw,code", [
    ("quantize", QUANT, dict(rows=-1), BAD), ("quantize", QUANT, dict(K=0), BAD), ("quantize", QUANT, dict(K=24), UNSUP),
    ("quantize", QUANT, dict(dtype=0), BAD), ("quantize", QUANT, dict(stride=63), BAD), ("quantize", QUANT, dict(x=None), BAD),
    ("quantize", QUANT, dict(x=FAKE + 1), BAD), ("quantize", QUANT, dict(codes=FAKE + 8), BAD), ("quantize", QUANT, dict(codes=None), BAD),
    ("quantize", QUANT, dict(scales=None), BAD), ("quantize", QUANT, dict(scales=FAKE + 2), BAD), ("quantize", QUANT, dict(rows=1 << 29), UNSUP),
    ("quantize_weights", SQUARES, dict(E=-1), BAD), ("quantize_weights", SQUARES, dict(rows=0), BAD), ("quantize_weights", SQUARES, dict(K=0), BAD),
    ("quantize_weights", SQUARES, dict(K=40), UNSUP), ("quantize_weights", SQUARES, dict(rows=40, transpose=1), UNSUP),
    ("quantize_weights", SQUARES, dict(E=65536), UNSUP), ("quantize_weights", SQUARES, dict(rows=(1 << 20) + 16), UNSUP),
    ("quantize_weights", SQUARES, dict(rows=1 << 20, K=1 << 20), UNSUP), ("quantize_weights", SQUARES, dict(dtype=7), BAD),
    ("quantize_weights", SQUARES, dict(x=None), BAD), ("quantize_weights", SQUARES, dict(codes=FAKE + 4), BAD), ("quantize_weights", SQUARES, dict(scales=None), BAD),
    ("dequantize", BACK, dict(rows=-1), BAD), ("dequantize", BACK, dict(K=8), UNSUP), ("dequantize", BACK, dict(dtype=0), BAD),
    ("dequantize", BACK, dict(codes=FAKE + 1), BAD), ("dequantize", BACK, dict(scales=FAKE + 1), BAD), ("dequantize", BACK, dict(out=None), BAD),
    ("dequantize", BACK, dict(rows=1 << 40), UNSUP),
    ("dequantize_weights", BACK_SQUARES, dict(E=-2), BAD), ("dequantize_weights", BACK_SQUARES, dict(rows=0), BAD), ("dequantize_weights", BACK_SQUARES, dict(K=56), UNSUP),
    ("dequantize_weights", BACK_SQUARES, dict(E=1 << 20), UNSUP), ("dequantize_weights", BACK_SQUARES, dict(codes=None), BAD), ("dequantize_weights", BACK_SQUARES, dict(out=FAKE + 1), BAD),
])
def test_conversions_refuse(name, defaults, kw, code):
    _refused("qmoe_blocks_" + name, defaults, kw, code)


PRODUCT = dict(a=FAKE, sa=FAKE, a_rows=8, w=FAKE, sw=FAKE, E=4, N=32, K=64, offsets=FAKE, routes=None, k=1, rows=8,
               dtype=2, out=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), BAD), (dict(E=1025), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=72), UNSUP), (dict(K=1 << 21), UNSUP),
    (dict(N=(1 << 20) + 1), UNSUP), (dict(rows=-1), BAD), (dict(rows=1 << 31), BAD), (dict(rows=1 << 24, a_rows=1 << 24), UNSUP),
    (dict(rows=9), BAD), (dict(a_rows=-1), BAD), (dict(a_rows=1 << 31), BAD), (dict(dtype=0), BAD), (dict(dtype=3), UNSUP), (dict(k=0), BAD),
    (dict(offsets=None), BAD), (dict(routes=FAKE, a_rows=1 << 26), UNSUP), (dict(routes=FAKE, a_rows=0), BAD),
    (dict(rows=1 << 23, a_rows=1 << 23, N=1 << 20), UNSUP), (dict(a=None), BAD), (dict(a=FAKE + 8), BAD), (dict(sa=None), BAD),
    (dict(sa=FAKE + 1), BAD), (dict(w=None), BAD), (dict(w=FAKE + 1), BAD), (dict(sw=None), BAD), (dict(offsets=FAKE + 2), BAD),
    (dict(routes=FAKE + 2), BAD), (dict(out=None), BAD), (dict(out=FAKE + 1), BAD),
])
def test_product_refuses(kw, code):
    _refused("qmoe_blocks_matmul", PRODUCT, kw, code)


ACT = dict(y=FAKE, stride=128, rows=4, I=64, dtype=1, act=0, fusion=1, alpha=1.0, beta=0.0, limit=INF)
FORMS = [("qmoe_activate", dict(ACT, out=FAKE, stream=None)),
         ("qmoe_activate_blocks", dict(ACT, codes=FAKE, scales=FAKE, stream=None)),
         ("qmoe_activate_backward", dict(grad=FAKE, gstride=64, **ACT, out=FAKE, stream=None))]


@pytest.mark.parametrize("name,defaults", FORMS)
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(I=0), BAD), (dict(I=(1 << 19) + 16), UNSUP), (dict(rows=1 << 40), UNSUP), (dict(dtype=0), BAD),
    (dict(act=2), BAD), (dict(fusion=0), BAD), (dict(fusion=3), BAD), (dict(alpha=NAN), BAD), (dict(beta=NAN), BAD),
    (dict(limit=NAN), BAD), (dict(limit=0.0), BAD), (dict(limit=-1.0), BAD), (dict(y=None), BAD), (dict(y=FAKE + 1), BAD),
    (dict(stride=127), BAD),
])
def test_activation_refuses(name, defaults, kw, code):
    _refused(name, defaults, kw, code)


def test_activation_outputs_are_checked():
    _refused(*FORMS[0], dict(out=None), BAD)
    _refused(*FORMS[0], dict(out=FAKE + 1), BAD)
    for kw, code in ((dict(codes=None), BAD), (dict(codes=FAKE + 8), BAD), (dict(scales=FAKE + 2), BAD), (dict(I=40), UNSUP)):
        _refused(*FORMS[1], kw, code)
    for kw in (dict(grad=None), dict(gstride=63), dict(grad=FAKE + 1), dict(out=None), dict(out=FAKE + 1)):
        _refused(*FORMS[2], kw, BAD)


def test_nothing_to_do_touches_nothing():
    for name, defaults, kw in (("qmoe_route_scores", ROUTE, dict(T=0, logits=None, ids=None, weights=None)),
                               ("qmoe_route_scores_backward", ROUTE_GRAD, dict(T=0, logits=None, out=None)),
                               ("qmoe_blocks_quantize", QUANT, dict(rows=0, x=None, codes=None)),
                               ("qmoe_blocks_quantize_weights", SQUARES, dict(E=0, x=None, codes=None)),
                               ("qmoe_blocks_dequantize", BACK, dict(rows=0, out=None)),
                               ("qmoe_blocks_dequantize_weights", BACK_SQUARES, dict(E=0, out=None)),
                               ("qmoe_blocks_matmul", PRODUCT, dict(rows=0, a=None, out=None)),
                               (*FORMS[0], dict(rows=0, y=None, out=None)), (*FORMS[1], dict(rows=0, y=None, codes=None)),
                               (*FORMS[2], dict(rows=0, y=None, grad=None, out=None))):
        assert _call(name, defaults, kw) == qm.OK, qm.last_error()
        assert qm.last_error() == ""


def test_binding_refuses_tensors_of_the_host():
    x, codes = torch.zeros(4, 64), torch.zeros(4, 64, dtype=qm.FP8_DTYPE)
    scales = torch.zeros(4, 1)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: qm.route_scores(x, 2), lambda: qm.route_scores_backward(x, x, ids), lambda: qm.fp8_quantize(x),
                 lambda: qm.fp8_quantize_weights(x), lambda: qm.fp8_dequantize(codes, scales, torch.float32),
                 lambda: qm.fp8_dequantize_weights(codes, scales, torch.float32),
                 lambda: qm.fp8_matmul(codes, scales, codes, scales), lambda: qm.activate(x), lambda: qm.activate_fp8(x),
                 lambda: qm.activate_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="top_k"):
        qm.fp8_matmul(codes, scales, codes, scales, sorted_routes=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("name,defaults", [("quantize", dict(QUANT, stride=1 << 31)), ("dequantize", BACK)])
@pytest.mark.parametrize("K", [(1 << 20) + 16, (1 << 31) - 16])  # the count of the longest row's blocks left 32 bits
def test_conversions_refuse_wider_rows(name, defaults, K):
    _refused("qmoe_blocks_" + name, defaults, dict(rows=1, K=K), UNSUP)
