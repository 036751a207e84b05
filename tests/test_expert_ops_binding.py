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


def test_shared_memory_is_found():
    # rows of a wide buffer: what lies between the first and the last element counts
    buf = torch.zeros(100)
    out = buf[40:60].view(4, 5)
    qm._apart(out, before=buf[:40], behind=buf[60:], strided=buf[:36].view(6, 6)[:, :2], none=None, empty=buf[50:50])
    for t in (buf, buf[59:], buf[:41], buf[45:46], buf.view(10, 10)[:5, :2]):
        with pytest.raises(ValueError, match="out overlaps it"):
            qm._apart(out, it=t)


@pytest.mark.gpu
def test_given_outputs_must_lie_apart():
    # in place, a workgroup's rows were overwritten before others had read them
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    rows, _, _, rr = qm.permute(torch.zeros((4, 64), device="cuda"), ids, 2)
    with pytest.raises(ValueError, match="overlaps rows"):
        qm.unpermute(rows, rr, out=rows[:4])
    with pytest.raises(ValueError, match="overlaps rows"):
        qm.permute_backward(rows, rr, out=rows[4:])
    both = torch.zeros((12, 64), device="cuda")
    assert qm.unpermute(both[:8], rr, out=both[8:]).eq(0).all()
    pool = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    codes, scales = pool[:128].view(4, 32), pool[128:136].view(4, 2)
    with pytest.raises(ValueError, match="overlaps scales"):
        qm.mx_dequantize(codes, scales, torch.float32, out=pool[128:1152].view(torch.float32).view(4, 64))
    with pytest.raises(ValueError, match="overlaps a_codes"):
        qm.mx_matmul(codes, scales, codes.clone(), scales.clone(), dtype=torch.float32,
                     out=pool[64:128].view(torch.float32).view(4, 4))
