"""The router with more tokens than the losses' small workgroups hold at once, for every number of lanes a token (MI355X).

From 131,072 lanes of tokens on, the losses' launch has workgroups of 16 waves, whose partial sums and selections fill
64 KB of LDS; tokens are 8, 16, 32 or 64 lanes wide. Checks and tolerances are those of test_gpu_router.py.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say
from test_gpu_router import DEV, check_backward, check_forward, check_losses, logits

pytestmark = pytest.mark.gpu


@pytest.mark.timeout(300)
@pytest.mark.parametrize("T,E,k,dtype,kind", [
    (17001, 1, 1, "f32", "normal"), (16385, 8, 2, "bf16", "masked"), (20001, 60, 4, "bf16", "normal"),
    (33000, 64, 8, "f32", "ties"), (8193, 100, 6, "bf16", "normal"), (9001, 128, 8, "f32", "masked"),
    (4097, 200, 4, "bf16", "normal"), (5001, 256, 16, "f32", "far"), (2049, 300, 5, "f32", "normal"),
    (2600, 512, 8, "bf16", "ties"), (2100, 1000, 64, "f32", "normal"),
])
def test_many_tokens(T, E, k, dtype, kind):
    say(f"[gpu] router wide batch T={T} E={E} k={k} {dtype} {kind}")
    x = logits(T, E, dtype, T + E, kind)
    xd = x.to(DEV)
    rng = np.random.default_rng(T)
    d_w, d_losses = rng.normal(size=(T, k)).astype(np.float32), np.array([0.25, -0.5], dtype=np.float32)
    renormalize = T % 2 == 0
    r = moe.moe_router_topk_losses(xd, k, renormalize=renormalize)
    ids, w, lse = check_forward(x, k, renormalize, r)
    counts, n = check_losses(x, ids, lse, r)
    d = moe.moe_router_backward(xd, r, torch.from_numpy(d_w).to(DEV), torch.from_numpy(d_losses).to(DEV))
    check_backward(x, dtype, ids, renormalize, d, d_w, d_losses, counts, n)
