"""Router gradient with counts summed over several ranks: the slots of all experts together pass 2^31 (on an MI355X).

The counts and tokens are those of a global batch, the logits one rank's part of it. Tolerances as in test_gpu_router.py:
the sum of the counts is a whole number and rounded once.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say
from oracle import router as orr
from test_gpu_router import DEV, check_backward, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k", [(5, 8, 2), (64, 65, 6), (9, 200, 4), (6, 512, 8), (3, 1024, 64)])
def test_counts_of_a_global_batch(T, E, k, dtype):
    say(f"[gpu] router gradient, counts of a global batch, T={T} E={E} k={k} {dtype}")
    rng = np.random.default_rng(E)
    x = logits(T, E, dtype, E, "normal")
    xd = x.to(DEV)
    n = 2 ** 30 + 7
    counts = rng.integers(0, min(2 ** 31 - 1, 2 * k * n // E), size=E).astype(np.int32)
    counts[0], counts[E - 1] = 0, 2 ** 31 - 1
    assert counts.astype(np.int64).sum() > 2 ** 31
    r = moe.moe_router_topk_losses(xd, k)
    r.counts.copy_(torch.from_numpy(counts))
    r.tokens.fill_(n)
    d_losses = np.array([0.25, -0.5], dtype=np.float32) * np.float32(2 ** 30)
    d = moe.moe_router_backward(xd, r, None, torch.from_numpy(d_losses).to(DEV))
    ids, _, _ = orr.topk(x.double().numpy(), k, True)
    check_backward(x, dtype, ids, True, d, None, d_losses.astype(np.float64), counts.astype(np.int64), n)
