"""The router's gradient against differences of the kernels' own weights and losses, every logit of every row (MI355X).

A row's logits are 1/4 apart and move by h = 1/16, so no probe changes a choice. Central differences are off by h^2 / 6
of the third derivative. With p the probability that moves: softmax's, of a sum with coefficients of spread s, is at most
s |p'''| <= s / 8 (p''' = p (1 - p) (1 - 6 p (1 - p))), of the weights s <= 2 max |g|, of the balance loss
s <= max c = E max f / n. That of lse^2 is 2 (3 p^2 (1 - p) + lse p (1 - p) (1 - 2 p)) <= 2 (4/9 + |lse| / 10).
The rounding of the two evaluations, over 2 h, is that which test_gpu_router.py derives for weights and losses; the
other rows' weights are the same bits in both. The gradient's own rounding is 200 u of its terms' sizes.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say
from test_gpu_router import DEV, U

pytestmark = pytest.mark.gpu

T, E, K, H = 3, 16, 4, 1.0 / 16
FAR = 15 / 4 + H


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_is_the_difference(renormalize):
    say(f"[gpu] router differences of every logit, renormalize={renormalize}")
    rng = np.random.default_rng(11)
    x = np.stack([rng.permutation(E) / 4 - 2 for _ in range(T)]).astype(np.float32)
    g = rng.normal(size=(T, K)).astype(np.float32)
    dl = np.array([1.0, 0.5], dtype=np.float32)

    def evaluate(v):
        r = moe.moe_router_topk_losses(torch.from_numpy(v).to(DEV), K, renormalize=renormalize)
        return r, (r.losses.cpu().numpy().astype(np.float64) * dl).sum() + (r.routing_w.cpu().numpy().astype(np.float64) * g).sum()

    r, _ = evaluate(x)
    d = moe.moe_router_backward(torch.from_numpy(x).to(DEV), r, torch.from_numpy(g).to(DEV), torch.from_numpy(dl).to(DEV))
    d = d.cpu().numpy().astype(np.float64)
    top = np.abs(g).max()
    f = r.counts.max().item() / (T * K)
    lse = 2 + H + np.log(E)
    third = 2 * top / 8 + dl[0] * E * f / T / 8 + dl[1] / T * 2 * (4 / 9 + lse / 10)
    chain = (T / 256 + 300) * U
    rounding = (top * (FAR + 40) * 2 * U + dl[0] * E * f * (chain + 220 * U + (E + 8) * U)
                + dl[1] * (2 * lse * (40 + lse) * 2 * U + lse * lse * (chain + 4 * U)))
    own = 200 * U * (2 * top + 2 * dl[0] * E * f / T + 2 * dl[1] * lse / T)
    tol = H * H / 6 * third + rounding / H + own
    compared = 0
    for t in range(T):
        for e in range(E):
            up, dn = x.copy(), x.copy()
            up[t, e] += H
            dn[t, e] -= H
            (ru, lu), (rd, ld) = evaluate(up), evaluate(dn)
            assert torch.equal(ru.expert_ids, r.expert_ids) and torch.equal(rd.expert_ids, r.expert_ids)
            assert abs((lu - ld) / (2 * H) - d[t, e]) <= tol, (t, e, (lu - ld) / (2 * H), d[t, e], tol)
            compared += 1
    assert compared == T * E
    assert np.abs(d).max() > 20 * tol  # a missing term would show
