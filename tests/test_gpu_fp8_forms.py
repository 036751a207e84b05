"""GPU tests of every form of the grouped product of e4m3 rows at its borders: short and ragged K, odd widths,
experts without rows, tiles that end early, rows behind the last expert."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_fp8 import _matmul_case

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16

# form, E, N, counts of rows by expert (a last extra one: dropped rows)
FORMS = [
    ("rows", 1, 70, [1]),
    ("rows", 4, 500, [3, 0, 17, 16, 5]),
    ("rows", 8, 33, [0, 0, 0, 0, 0, 0, 0, 2]),
    ("rows32", 1, 4100, [3]),
    ("rows32", 9, 800, [1, 0, 2, 9, 3, 1, 0, 0, 5, 4]),
    ("rows32", 2, 2050, [17, 30]),
    ("32x64", 1, 2049, [130]),
    ("32x64", 3, 1000, [33, 0, 95]),
    ("32x64", 40, 200, [1] * 30 + [0] * 9 + [7, 4]),
    ("64x128", 5, 3700, [64, 1, 0, 70, 20]),
    ("64x128", 300, 130, [2] * 150 + [0] * 149 + [90, 3]),
    ("64x128", 1, 4000, [500]),
    ("128x128", 2, 2100, [1001, 3]),
    ("128x128", 3, 2049, [0, 900, 260, 40]),
    ("256x256", 1, 4100, [2100]),
    ("256x256", 2, 4095, [1500, 900, 13]),
]


@pytest.mark.parametrize("K", [16, 128, 144, 256, 400, 640])
@pytest.mark.parametrize("form,E,N,counts", FORMS)
def test_forms(form, E, N, counts, K):
    if form == "256x256" and K not in (144, 256, 400):
        return
    _matmul_case(sum(counts), 1, E, K, N, BF16 if K % 128 else F16, K % 256 != 0, K + N, counts=counts)
