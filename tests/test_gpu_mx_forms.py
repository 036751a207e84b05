"""GPU tests of the grouped MXFP4 product's forms: every tile shape, with scales by either path."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _poisoned(t):
    """The same bytes between neighbours of 0xff: NaN scales, and codes of -6."""
    buf = torch.full((t.numel() + 512,), 255, dtype=torch.uint8, device="cuda")
    buf[256:256 + t.numel()] = t.reshape(-1)
    return buf[256:256 + t.numel()].view(t.shape)


def _operand(g, *shape):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(115, 125, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda").to(torch.uint8)
    return _poisoned(codes), _poisoned(scales)


def _offsets(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).int()


# E, K, N, rows of each expert, gather: K that ends behind half a group of steps, whose last scale row has 16
# bytes of the 32 that a group loads; the shortest rows; fewer columns and rows than a tile
@pytest.mark.parametrize("E,K,N,counts,gather", [
    (1, 32, 1, [1], False), (2, 96, 3, [1, 2], True), (1, 1024, 17, [5], False),
    (1, 1536, 33, [40], False), (3, 1536, 100, [9, 0, 60], True), (8, 1536, 4100, [130, 1, 255, 0, 129, 256, 7, 125], True),
    (2, 1536, 16410, [2000, 2390], False), (1, 3584, 12300, [4300], True),
])
def test_neighbours_of_the_operands_do_not_matter(E, K, N, counts, gather):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    rows = sum(counts)
    a, w = _operand(g, rows, K), _operand(g, E, N, K)
    routes = torch.randperm(rows, generator=g, device="cuda").int() if gather else None
    out = qm.mx_matmul(*a, *w, _offsets(counts), sorted_routes=routes, top_k=1, dtype=BF16)
    clean = qm.mx_matmul(*(t.clone() for t in (*a, *w)), _offsets(counts), sorted_routes=routes, top_k=1, dtype=BF16)
    assert not bool(torch.isnan(out).any())
    assert torch.equal(out, clean)


@pytest.mark.parametrize("rows,N,K", [(64, 40, 96), (600, 300, 1536)])
def test_decreasing_offsets_stay_inside_the_output(rows, N, K):
    # every second expert spans all rows: more tiles than any table that does not decrease can make
    g = torch.Generator(device="cuda").manual_seed(rows)
    E = 64
    a, w = _operand(g, rows, K), _operand(g, E, N, K)
    off = torch.tensor([0, rows] * (E // 2) + [rows], dtype=torch.int32, device="cuda")
    buf = torch.full((rows + 2, N), 7.0, device="cuda")
    qm.mx_matmul(*a, *w, off, dtype=F32, out=buf[1:rows + 1])
    assert buf[0].eq(7).all() and buf[-1].eq(7).all()
