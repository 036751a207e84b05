"""Sizes that do not fit the 32 bits in which the library takes them are refused by the binding: ctypes
passes the low bits, so 2^32 + 8 experts ran as 8, and a row of 2^32 + 32 values was quantised as 32."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm

WIDE = 1 << 32


def test_workspace_size_refuses_wide_sizes():
    for args in ((8, 2, WIDE + 8), (8, WIDE + 2, 8), (8, 2, 8 - WIDE), (8, 2, 1 << 31)):
        with pytest.raises(qm.QMoEError) as e:
            qm.permute_workspace_size(*args)
        assert e.value.code == qm.ERR_UNSUPPORTED
    assert qm.permute_workspace_size(8, 2, -1) == 0  # what fits is left to the library


@pytest.mark.gpu
def test_calls_refuse_wide_sizes():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    codes = torch.zeros((4, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    order = torch.arange(4, dtype=torch.int32, device="cuda")
    long_row = torch.empty(WIDE + 32, dtype=torch.float16, device="cuda")
    long_codes = torch.empty(WIDE // 2 + 16, dtype=torch.uint8, device="cuda")
    long_scales = torch.empty(WIDE // 32 + 1, dtype=torch.uint8, device="cuda")
    wide = long_row.view(1, -1)
    one = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: qm.permute(None, ids, WIDE + 8), lambda: qm.permute(None, ids, 8 - WIDE),
                 lambda: qm.permute(wide, one, 1), lambda: qm.unpermute(wide, one),
                 lambda: qm.unpermute_backward(wide, None, one),
                 lambda: qm.mx_quantize(long_row), lambda: qm.mx_quantize(wide),
                 lambda: qm.mx_quantize(long_row.view(-1, 1), transpose=True),
                 lambda: qm.mx_dequantize(long_codes, long_scales, torch.float16),
                 lambda: qm.mx_matmul(codes, scales, codes, scales, sorted_routes=order, top_k=WIDE + 1),
                 lambda: qm.mx_matmul(long_codes.view(1, -1), long_scales.view(1, -1), long_codes.view(1, -1),
                                      long_scales.view(1, -1))):
        with pytest.raises(qm.QMoEError) as e:
            call()
        assert e.value.code == qm.ERR_UNSUPPORTED
