"""GPU tests of the grouped MXFP4 product with scales far apart: large against small, the whole range of the
byte, and zeros under the largest scales."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _operand(rng, rows, K, lo, hi):
    return (rng.integers(0, 256, (rows, K // 2), dtype=np.uint8),
            rng.integers(lo, hi, (rows, K // 32), dtype=np.uint8))


# scale bytes of a and of w, [lo, hi): their products near 1, or (the last) anywhere
@pytest.mark.parametrize("a_range,w_range", [((240, 255), (0, 15)), ((0, 15), (240, 255)), ((254, 255), (0, 1)),
                                             ((0, 1), (254, 255)), ((247, 248), (7, 8)), ((0, 255), (0, 255))])
@pytest.mark.parametrize("rows,K,N,dtype", [(33, 32, 96, F32), (1, 64, 40, BF16), (70, 1024, 200, F32), (300, 96, 520, F16),
                                            (600, 1536, 300, BF16)])
def test_scales_far_apart(rows, K, N, dtype, a_range, w_range):
    rng = np.random.default_rng(rows + K + a_range[0])
    a, w = _operand(rng, rows, K, *a_range), _operand(rng, N, K, *w_range)
    got = qm.mx_matmul(*(torch.from_numpy(v).cuda() for v in (*a, *w)), dtype=dtype).double().cpu().numpy()
    av, wv = ref.values(*a), ref.values(*w)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv.T)
    # products of two codes are exact; K roundings (or truncations: 2 U32 each) of partial sums no larger than
    # mag; terms and sums below float32's normal range may count as zero; then one rounding to the type
    acc = K * 2 * ref.U32 * mag + K * 2.0 ** -126
    tol = acc + ref.HALF_STEP[dtype] * (np.abs(want) + acc) + ref.HALF_MIN[dtype]
    inside = (np.abs(want) + tol < torch.finfo(dtype).max) & (mag < torch.finfo(F32).max)
    # scales that differ by the whole range leave float32 in long sums, and float16 often
    assert inside.any() and (a_range == (0, 255) or inside.mean() > 0.9 or dtype == F16)
    assert np.all(np.abs(got - want)[inside] <= tol[inside])


@pytest.mark.parametrize("rows,K,N", [(5, 32, 40), (70, 1024, 200), (600, 1536, 300)])
def test_zeros_under_the_largest_scales(rows, K, N):
    rng = np.random.default_rng(rows)
    wc, ws = _operand(rng, N, K, 254, 255)
    zero = rng.choice(np.array([0x00, 0x08, 0x80, 0x88], dtype=np.uint8), (rows, K // 2))  # zeros of both signs
    for byte in (0, 127, 254):
        sa = np.full((rows, K // 32), byte, dtype=np.uint8)
        out = qm.mx_matmul(*(torch.from_numpy(v).cuda() for v in (zero, sa, wc, ws)), dtype=F32)
        assert out.eq(0).all()
