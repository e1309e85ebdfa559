"""The measured HBM traffic in bench.py's line: given while the profiled kernel's code is the tree's, and only then."""

import json
import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def test_the_committed_profile_is_of_this_code():
    """If this fails the gate/up kernel's code has changed: take profiles/zipf64_hbm_traffic.md's two runs again."""
    with open(bench.TRAFFIC_FILE) as f:
        tr = json.load(f)
    assert bench.measured_traffic("zipf64", True) == tr["bytes_per_launch"] > bench.algorithmic_bytes(
        8192, 8, 65536, 2048, 768, 60, fused=True)["gemm_up_swiglu"]
    assert bench.measured_traffic("zipf64", False) is None and bench.measured_traffic("square", True) is None


@pytest.mark.parametrize("name", ["gemm.hip", "grouped.h", "common.h"])
def test_every_source_of_the_kernel_counts(name, tmp_path, monkeypatch):
    names = [os.path.basename(p) for p in bench.kernel_sources(bench.GEMM_SRC)]
    assert names == ["gemm.hip", "grouped.h", "common.h"]
    for p in bench.kernel_sources(bench.GEMM_SRC):
        shutil.copy(p, tmp_path)
    monkeypatch.setattr(bench, "GEMM_SRC", str(tmp_path / "gemm.hip"))
    assert bench.measured_traffic("zipf64", True) is not None
    src = tmp_path / name
    text = src.read_text()
    src.write_text("// a comment\n" + text + "/* another\n one */\nhipError_t launch_something(const uint16_t* x,\n    int n);\n")
    assert bench.measured_traffic("zipf64", True) is not None
    src.write_text(text + "\nconstexpr int kMore = 1;\n")
    assert bench.measured_traffic("zipf64", True) is None
