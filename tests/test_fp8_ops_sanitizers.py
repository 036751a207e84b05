"""The host code of routing by scores, of the 8-bit floating point operators and of the gated activation
(fp8_ops.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, with the launchers replaced by the
stand-ins in tests/sanitize/fp8_ops_check.cpp.  No GPU is involved."""
import os
import subprocess

import pytest

from tests.test_host_sanitizers import CLANG, FLAGS, ROOT

SOURCES = [os.path.join(ROOT, "quantized_mixture_experts_route_amd", "csrc", "qmoe_api.cpp"),
           os.path.join(ROOT, "quantized_mixture_experts_route_amd", "csrc", "fp8_ops.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "stubs.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "fp8_ops_check.cpp")]


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang++ not installed")
def test_fp8_ops_host_code_clean_under_asan_and_ubsan(tmp_path):
    objs = []
    for src in SOURCES:
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        res = subprocess.run([CLANG, *FLAGS, "-c", src, "-o", obj], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
        objs.append(obj)
    exe = str(tmp_path / "fp8_ops_check")
    res = subprocess.run([CLANG, "-fsanitize=address,undefined", *objs, "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1:detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-6000:]
    assert "checks passed" in res.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
