"""Arguments of the sort by expert and of the MXFP4 operators that only make sense together."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm


def test_matmul_routes_need_their_top_k():
    # with an assumed top_k of 1, the routes of a top-k sort read wrong tokens or none, and nothing said so
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    order = torch.arange(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="top_k"):
        qm.mx_matmul(codes, scales, codes, scales, sorted_routes=order)


@pytest.mark.gpu
def test_matmul_takes_rows_by_name_and_by_route():
    g = torch.Generator(device="cuda").manual_seed(0)
    a, w = qm.mx_quantize(torch.randn(5, 64, generator=g, device="cuda")), qm.mx_quantize(torch.randn(7, 64, generator=g, device="cuda"))
    plain = qm.mx_matmul(*a, *w)
    with pytest.raises(ValueError, match="top_k"):
        qm.mx_matmul(*a, *w, sorted_routes=torch.arange(5, dtype=torch.int32, device="cuda"))
    named = torch.tensor([4, 0, 0, 2, 3, 1, 4], dtype=torch.int32, device="cuda")
    assert torch.equal(qm.mx_matmul(*a, *w, sorted_routes=named, top_k=1), plain[named.long()])
    routes = torch.tensor([9, 8, 1, 0, 5], dtype=torch.int32, device="cuda")
    assert torch.equal(qm.mx_matmul(*a, *w, sorted_routes=routes, top_k=2), plain[routes.long() // 2])
