"""The binding imports, and refuses CPU tensors, on a torch without a GPU backend."""

import os
import subprocess
import sys

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import ragged_grouped_gemm_histogram_amd as moe
assert moe.header_functions()
try:
    moe.moe_router_topk(torch.zeros((4, 8)), 2)
except ValueError as e:
    print("refused:", e)
"""


def test_import_without_a_gpu_backend():
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.startswith("refused: logits must be on"), res.stdout


@pytest.mark.gpu
def test_both_stream_queries_agree():
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert moe._public_stream(0) == moe._raw_stream(0) == s.cuda_stream
