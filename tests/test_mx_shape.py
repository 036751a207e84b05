"""The arithmetic behind the grouped MXFP4 product's loads and tiles (csrc/mx_shape.h), on the host."""
import os
import re
import subprocess

import pytest

import quantized_mixture_experts_route_amd as qm
from tests.test_gpu_mx_forms import FORMS
from tests.test_host_sanitizers import CLANG, FLAGS, ROOT

CSRC = os.path.join(ROOT, "quantized_mixture_experts_route_amd", "csrc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not installed")
    tmp = tmp_path_factory.mktemp("mx_shape")
    obj, exe = str(tmp / "check.o"), str(tmp / "check")
    for cmd in ([CLANG, *FLAGS, "-c", os.path.join(ROOT, "tests", "sanitize", "mx_shape_check.cpp"), "-o", obj],
                [CLANG, "-fsanitize=address,undefined", obj, "-o", exe]):
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
    return exe


def test_shape_arithmetic(checker):
    res = subprocess.run([checker], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "checks passed" in res.stdout, res.stdout + res.stderr


def test_loads_to_lds_carry_their_whole_offset_in_the_lane():
    # the descriptor starts at the step and the scalar offset is 0: with the step in the scalar offset, the
    # last scale row of an odd half group, and a step behind the last tile, were kept inside only by how the
    # hardware adds that offset to its range comparison
    text = open(os.path.join(CSRC, "mx_matmul.hip")).read()
    calls = re.findall(r"raw_ptr_buffer_load_lds\(([^;]*)\);", text)
    assert len(calls) == 1
    offset, immediate, aux = (v.strip() for v in calls[0].split(",")[-3:])
    assert (offset, immediate, aux) == ("0", "0", "0")
    assert "mx_bytes_left(bytes, at)" in text


def test_items_are_bounded_before_the_search():
    # a decreasing table of 1024 experts over 65536 rows of 2^20 columns makes 2^32 items: the count wrapped
    text = open(os.path.join(CSRC, "mx_matmul.hip")).read()
    assert re.search(r"const int total = mx_items\(first\[a\.E\], n_tiles, a\.rows, BM, a\.E\);", text)


def test_more_outputs_than_items_count_are_refused():
    fake = 1 << 20
    rc = qm.load_library().qmoe_mx_matmul(fake, fake, 1 << 23, fake, fake, 1, 1 << 20, 32, None, None, 1, 1 << 23, 2,
                                          fake, None)
    assert rc == qm.ERR_UNSUPPORTED and "2^40" in qm.last_error()


def test_every_form_has_a_case(checker):
    lines = "".join(f"{E} {N} {K} {sum(counts)}\n" for _, E, K, N, counts in FORMS)
    res = subprocess.run([checker, "forms"], input=lines, capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    assert res.stdout.splitlines() == [f[0] for f in FORMS]
    tiles = ["32x64s4", "64x128s4", "128x128s4"]
    want = {f"{t} {p} full" for t in tiles for p in ("direct", "registers")}
    want |= {f"{t} {p} {h}" for t in ("64x128s2", "128x128s2", "256x256s2") for p in ("direct", "registers")
             for h in ("full", "half")}
    assert {f[0] for f in FORMS} == want
    # 16-bit rows that start between two words take stores of their own: an odd width for every tile
    assert {f[0].split()[0] for f in FORMS if f[3] % 2} == {w.split()[0] for w in want}
