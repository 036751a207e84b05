"""GPU tests of the grouped MXFP4 product's forms: every tile shape, with scales by either path."""
from __future__ import annotations

import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _expert_ref as ref

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


# Every form of the kernel: tile and stages, scales by the direct path or through registers, whether a half
# group of steps ends a tile (tests/test_mx_shape.py holds the names against the launch rule), with even and
# odd widths; E, K, N and the rows of each expert
FORMS = [
    ("32x64s4 direct full", 3, 2048, 200, [40, 0, 33]),
    ("32x64s4 direct full", 40, 2048, 129, [3, 1, 0, 9] * 10),
    ("32x64s4 registers full", 1, 1056, 127, [70]),
    ("64x128s4 direct full", 1, 4096, 4095, [512]),
    ("64x128s4 direct full", 4, 2048, 3500, [130, 128, 1, 200]),
    ("64x128s4 registers full", 1, 4128, 4001, [500]),
    ("128x128s4 direct full", 1, 4096, 3000, [1024]),
    ("128x128s4 direct full", 2, 2048, 3001, [255, 769]),
    ("128x128s4 registers full", 1, 4128, 3001, [1024]),
    ("64x128s2 direct full", 5, 1024, 300, [64, 1, 0, 65, 63]),
    ("64x128s2 direct full", 16, 2048, 8193, [50, 64, 1, 65, 63, 40, 0, 90] * 2),
    ("64x128s2 direct half", 16, 1536, 8193, [50, 64, 1, 65, 63, 40, 0, 90] * 2),
    ("64x128s2 registers full", 3, 288, 301, [64, 0, 90]),
    ("64x128s2 registers half", 16, 1312, 8190, [50, 64, 1, 65, 63, 40, 0, 90] * 2),
    ("128x128s2 direct full", 8, 2048, 4097, [128, 1, 255, 130, 0, 256, 129, 125]),
    ("128x128s2 direct half", 8, 1536, 4099, [128, 1, 255, 130, 0, 256, 129, 125]),
    ("128x128s2 registers full", 8, 1824, 4096, [128, 1, 255, 130, 0, 256, 129, 125]),
    ("128x128s2 registers half", 8, 1312, 4101, [128, 1, 255, 130, 0, 256, 129, 125]),
    ("256x256s2 direct full", 1, 2048, 10001, [4100]),       # several tiles a workgroup, rows between words
    ("256x256s2 direct full", 3, 1024, 16400, [1100, 0, 3000]),
    ("256x256s2 direct half", 2, 1536, 10003, [1900, 2300]),
    ("256x256s2 registers full", 2, 992, 16401, [1100, 3000]),
    ("256x256s2 registers half", 1, 1312, 10002, [4100]),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("form,E,K,N,counts", FORMS)
def test_every_form(form, E, K, N, counts, dtype, gather):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    k = 2 if gather else 1
    rows = sum(counts)
    a, w = _operand(g, -(-rows // k), K), _operand(g, E, N, K)
    routes = torch.randperm(rows, generator=g, device="cuda").int() if gather else None
    off = _offsets(counts)
    # out starts one element into a buffer: two bytes behind a word for the 16-bit types
    buf = torch.full((rows * N + 2,), 7.0, dtype=dtype, device="cuda")
    out = qm.mx_matmul(*a, *w, off, sorted_routes=routes, top_k=k, dtype=dtype, out=buf[1:-1].view(rows, N))
    assert buf[0] == 7 and buf[-1] == 7
    assert torch.equal(out, qm.mx_matmul(*a, *w, off, sorted_routes=routes, top_k=k, dtype=dtype))
    av = qm.mx_dequantize(*a, F32).double()
    av = av[routes.long() // k] if gather else av
    lo = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        wt = qm.mx_dequantize(w[0][e], w[1][e], F32).double().T.contiguous()
        want, mag = av[lo:lo + n] @ wt, av[lo:lo + n].abs() @ wt.abs()
        # products of scaled codes are exact; K roundings (or truncations: 2 U32 each) of partial sums no larger
        # than mag, then one rounding to the type
        acc = K * 2 * ref.U32 * mag
        tol = acc + ref.HALF_STEP[dtype] * (want.abs() + acc) + ref.HALF_MIN[dtype]
        assert bool(((out[lo:lo + n].double() - want).abs() <= tol).all()), (form, e)
        lo += n
