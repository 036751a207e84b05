"""GPU tests of the way back's gradient with many tokens: on both sides of the number of workgroups from which
bfloat16 rows are taken one slot at a time (1536 of them: 256 threads, a token's share of them a power of two)."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _strided(x, strided):
    if not strided:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + 5), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 3:-2] = x
    return wide[:, 3:-2]


# T, H, k: a workgroup a token, two, four, 16 and 32 tokens a workgroup, rows shorter than a vector
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,H,k,strided", [
    (1536, 2048, 2, False), (1537, 2051, 3, True), (2100, 1300, 1, False), (3500, 1001, 6, True),
    (6200, 300, 4, False), (26000, 72, 5, True), (50000, 24, 2, False), (60000, 5, 3, True),
])
def test_unpermute_backward_many_tokens(T, H, k, strided, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    E = 7
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda").int()  # an eighth of the routes is dropped
    rr = qm.permute(None, ids, E)[3]
    rows = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    grad = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = torch.randn(T, k, generator=g, device="cuda")
    got, got_w = qm.unpermute_backward(_strided(grad, strided), _strided(rows, strided), rr, w)
    only = qm.unpermute_backward(_strided(grad, strided), None, rr, w)[0]
    kept = rr >= 0
    at = torch.where(kept, rr, -1 - rr).long()
    # a kept route's row holds w * grad rounded once in float32 and once to the type; a dropped one's zeros
    for s in range(k):
        want = torch.where(kept[:, s:s + 1], w[:, s:s + 1].double() * grad.double(), 0.0)
        tol = (ref.U32 + ref.HALF_STEP[dtype]) * 1.01 * want.abs() + ref.HALF_MIN[dtype]
        assert bool(((got[at[:, s]].double() - want).abs() <= tol).all())
        terms = grad.double() * rows[at[:, s]].double() * kept[:, s:s + 1]
        # H float32 roundings at most of partial sums no larger than the sum of magnitudes
        assert bool(((got_w[:, s].double() - terms.sum(1)).abs() <= (H + 1) * ref.U32 * terms.abs().sum(1)).all())
    assert torch.equal(only, got)
    again = qm.unpermute_backward(_strided(grad, strided), _strided(rows, strided), rr, w)
    assert torch.equal(again[0], got) and torch.equal(again[1], got_w)
