"""Traffic counters of the layer stay valid while only the operators beside it change."""
from __future__ import annotations

import glob
import os
import re
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "quantized_mixture_experts_route_amd", "csrc")


def test_digest_leaves_out_what_no_layer_kernel_includes():
    names = {os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*"))}
    assert set(bench.OTHER_OPERATORS) <= names
    for name in sorted(names - set(bench.OTHER_OPERATORS)):
        if not name.endswith(".cpp"):  # qmoe_api.cpp takes one declaration from expert_ops.h
            included = set(re.findall(r'#include "([^"]+)"', open(os.path.join(CSRC, name)).read()))
            assert not included & set(bench.OTHER_OPERATORS), name


def test_digest_follows_the_layers_sources_alone(tmp_path, monkeypatch):
    copy = tmp_path / "quantized_mixture_experts_route_amd" / "csrc"
    shutil.copytree(CSRC, copy)
    before = bench.kernel_source_digest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_digest() == before
    for name in bench.OTHER_OPERATORS:
        with open(copy / name, "a") as f:
            f.write("// changed\n")
    assert bench.kernel_source_digest() == before
    with open(copy / "gemm_prefill.hip", "a") as f:
        f.write("// changed\n")
    assert bench.kernel_source_digest() != before
