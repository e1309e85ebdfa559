"""Pins of the 64-bit router and MXFP4 references: autograd, differences, and the format's printed values (no GPU)."""

import numpy as np
import pytest
import torch

from oracle import mxfp4 as om
from oracle import router as orr


def _case(seed, T=7, E=9, masked=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)) * 2
    if masked:
        x[0, :] = -np.inf
        x[1, 2:] = -np.inf
        x[2, [0, 4]] = -np.inf
    return rng, x


@pytest.mark.parametrize("renormalize", [False, True])
def test_router_backward_is_autograd_of_the_forward(renormalize):
    rng, x = _case(1)
    k = 4
    ids, w, lse = orr.topk(x, k, renormalize)
    counts, n, P, L = orr.losses(x, ids)
    g, dl = rng.normal(size=(7, k)), np.array([0.3, -0.2])
    live = ~np.isneginf(lse)
    t = torch.tensor(x[live], requires_grad=True)
    p = torch.softmax(t, 1)
    kept = torch.tensor(ids[live] >= 0)
    pk = torch.gather(p, 1, torch.tensor(ids[live]).clamp(min=0).long()) * kept
    tw = pk / pk.sum(1, keepdim=True) if renormalize else pk
    np.testing.assert_allclose(tw.detach().numpy(), w[live], rtol=1e-12, atol=1e-300)
    E = x.shape[1]
    f = torch.tensor(counts / counts.sum())
    balance = E * (f * p.sum(0) / n).sum()
    z = (torch.logsumexp(t, 1) ** 2).sum() / n
    np.testing.assert_allclose([balance.item(), z.item()], L, rtol=1e-12)
    (dl[0] * balance + dl[1] * z + (tw * torch.tensor(g[live])).sum()).backward()
    d, size = orr.backward(x, ids, renormalize, g, dl, counts, n)
    np.testing.assert_allclose(d[live], np.nan_to_num(t.grad.numpy()), rtol=1e-10, atol=1e-14)
    assert not d[~live].any() and (np.abs(d) <= size + 1e-300).all()


def test_router_backward_is_the_difference_of_the_loss():
    rng, x = _case(2, masked=False)
    ids, _, _ = orr.topk(x, 3, True)
    g, dl = rng.normal(size=(7, 3)), np.array([0.7, 0.1])
    counts, n, _, _ = orr.losses(x, ids)

    def loss(v):
        i, w, _ = orr.topk(v, 3, True)
        assert (i == ids).all()
        return (dl * orr.losses(v, i)[3]).sum() + (g * w).sum()

    d, _ = orr.backward(x, ids, True, g, dl, counts, n)
    for t, e in [(0, 0), (3, 5), (6, 8), (2, int(ids[2, 0]))]:
        v = x.copy()
        v[t, e] += 1e-6
        u = x.copy()
        u[t, e] -= 1e-6
        assert abs((loss(v) - loss(u)) / 2e-6 - d[t, e]) < 1e-7


def test_topk_ties_masks_and_padding():
    inf = np.inf
    x = np.array([[1.0, 3.0, 3.0, 1.0], [-inf, -inf, 2.0, -inf], [-inf] * 4, [-3e38] * 4])
    ids, w, lse = orr.topk(x, 3, False)
    assert ids.tolist() == [[1, 2, 0], [2, -1, -1], [-1, -1, -1], [0, 1, 2]]
    assert w[1].tolist() == [1.0, 0.0, 0.0] and not w[2].any() and lse[2] == -inf
    assert w[3].tolist() == [0.25] * 3
    counts, n, P, L = orr.losses(np.zeros((6, 4)), np.arange(12).reshape(6, 2) % 4)
    assert counts.tolist() == [3] * 4 and n == 6 and L[0] == 1.0  # both uniform


def test_mxfp4_grid_ties_and_saturation():
    # halfway points go to the even code; past 6 everything is 6
    y = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7.9])
    assert om.GRID[om.nearest_code(y)].tolist() == [0, 0, 0.5, 1, 1, 2, 2, 3, 4, 4, 6, 6]


def test_mxfp4_blocks():
    x = np.zeros((2, 40))
    x[0, 0], x[0, 1], x[0, 39] = 7.0, -1.0, 2.0 ** -126
    x[1, 5], x[1, 33] = np.nan, 2.0 ** -133
    q, s = om.quantize(x)
    assert q.shape == (2, 32) and s.shape == (2, 16)
    assert s[0, :3].tolist() == [127, 0, 0] and s[1, :2].tolist() == [255, 0]
    v = om.dequantize(q, s, 40)
    assert v[0, 0] == 6.0 and v[0, 1] == -1.0 and v[0, 39] == 2.0 ** -126
    assert np.isnan(v[1, :32]).all() and v[1, 33] == 0.0  # 2^-133 is 2^-6 of the least scale: below half a step
    # every code reads back as itself
    codes = np.arange(16, dtype=np.uint8)
    row = np.concatenate([codes, codes])
    q = row[0::2] | (row[1::2] << 4)
    v = om.dequantize(q[None], np.full((1, 16), 130, np.uint8), 32)
    assert v[0, :16].tolist() == [g * 8 for g in om.GRID] + [-g * 8 for g in om.GRID]
    assert (om.quantize(v)[0] == q).all()
