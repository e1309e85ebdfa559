"""Router kernels against the 64-bit reference, on an MI355X.

Tolerances, all from fp32 arithmetic with u = 2^-24. An exponential's argument x - m is rounded once, so
exp(x - m) is off by (|x - m| + 2) u relative; the row sum of positive terms adds at most 32 roundings and carries its
terms' errors, weighted by e^-|x-m| (at most ln E <= 7 of them): p and w are off by (|x - m| + 60) u, taken as
(|x - m| + 40) 2 u. lse adds the logarithm's and the sum's rounding: (40 + |lse|) 2 u absolute. Column sums over T rows
run through chains of at most T / 256 + 300 additions of positive terms. A gradient is a sum of a few products: it is
off by (|x_i - m| + 96) 2 u of the magnitudes of its terms, plus half a step of the output's type.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say
from oracle import router as orr

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def logits(T, E, dtype, seed, kind):
    """float64 values of the type: normals with ties, masked experts, padded rows, the lowest value, a far offset."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)) * 2
    if kind == "ties":
        x = np.round(x)
    if kind == "far":
        x = x * 8 + 1000.0
    t = torch.from_numpy(x).to(DT[dtype])
    if kind == "masked":
        low = torch.finfo(DT[dtype]).min
        for r in range(T):
            if r % 5 == 0:
                t[r] = -np.inf
            elif r % 5 == 1:
                t[r, rng.permutation(E)[: max(0, E - 2)]] = -np.inf
            elif r % 5 == 2:
                t[r, rng.permutation(E)[: E // 2]] = low
            elif r % 5 == 3:
                t[r] = low
    return t


def check_forward(x, k, renormalize, r):
    X = x.double().numpy()
    ids, w, lse = orr.topk(X, k, renormalize)
    np.testing.assert_array_equal(r.expert_ids.cpu().numpy(), ids)
    top = X.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(ids >= 0, np.abs(np.take_along_axis(X, np.maximum(ids, 0).astype(np.int64), 1) - top), 0.0)
    far = np.minimum(np.nan_to_num(far, posinf=0.0), 200.0)  # beyond, the exponential is 0 in fp32
    err = np.abs(r.routing_w.cpu().numpy().astype(np.float64) - w)
    assert (err <= w * (far + 40) * 2 * U + 2.0 ** -126).all(), err.max()
    got = r.lse.cpu().numpy().astype(np.float64)
    live = ~np.isneginf(lse)
    assert np.isneginf(got[~live]).all()
    assert (np.abs(got[live] - lse[live]) <= (40 + np.abs(lse[live])) * 2 * U).all()
    return ids, w, lse


def check_losses(x, ids, lse, r):
    X = x.double().numpy()
    counts, n, P, L = orr.losses(X, ids)
    np.testing.assert_array_equal(r.counts.cpu().numpy(), counts)
    assert r.tokens.item() == n
    chain = (x.shape[0] / 256 + 300) * U
    far = 110 * 2 * U  # a term 70 below the maximum is below u of any column sum that holds a larger one
    tol = P * (chain + far) + 1e-30
    assert (np.abs(r.prob_mean.cpu().numpy() - P) <= tol).all()
    live = ~np.isneginf(lse)
    z_err = (2 * np.abs(lse[live]) * (40 + np.abs(lse[live])) * 2 * U).sum() / max(1, n) + L[1] * (chain + 4 * U)
    got = r.losses.cpu().numpy().astype(np.float64)
    assert abs(got[0] - L[0]) <= L[0] * (chain + far + (x.shape[1] + 8) * U)
    if L[1] > np.finfo(np.float32).max:  # lse near the type's lowest value: its square is past fp32's range
        assert np.isposinf(got[1])
    else:
        assert abs(got[1] - L[1]) <= z_err + 1e-30
    return counts, n


def check_backward(x, dtype, ids, renormalize, d, d_w, d_losses, counts, n):
    X = x.double().numpy()
    want, size = orr.backward(X, ids, renormalize, d_w, d_losses, counts, n)
    with np.errstate(invalid="ignore"):
        far = np.minimum(np.nan_to_num(np.abs(X - X.max(axis=1, keepdims=True)), posinf=0.0), 200.0)
    tol = size * (far + 96) * 2 * U + (np.abs(want) + size * 1e-4) * HALF[dtype] + 2.0 ** -126
    err = np.abs(d.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (4, 128, 8), (37, 64, 8), (64, 65, 6), (100, 100, 6), (257, 128, 8), (33, 200, 4),
          (17, 256, 16), (9, 300, 3), (20, 512, 8), (5, 513, 7), (4, 1000, 64), (3, 1024, 64), (4099, 64, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "far"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_router(T, E, k, kind, dtype):
    if T > 1000 and kind in ("ties", "far"):
        T = 700
    say(f"[gpu] router T={T} E={E} k={k} {kind} {dtype}")
    x = logits(T, E, dtype, 100 * T + E, kind)
    xd = x.to(DEV)
    rng = np.random.default_rng(T + E)
    d_w = rng.normal(size=(T, k)).astype(np.float32)
    d_losses = np.array([0.25, -0.5], dtype=np.float32)
    for renormalize in (True, False):
        r = moe.moe_router_topk(xd, k, renormalize=renormalize)
        ids, w, lse = check_forward(x, k, renormalize, r)
        tr = moe.moe_router_topk_losses(xd, k, renormalize=renormalize)
        for a, b in ((r.expert_ids, tr.expert_ids), (r.routing_w, tr.routing_w), (r.lse, tr.lse)):
            assert torch.equal(a, b)
        counts, n = check_losses(x, ids, lse, tr)
        dw = torch.from_numpy(d_w).to(DEV)
        dw[tr.expert_ids < 0] = float("nan")  # what a dropped slot holds does not matter
        dl = torch.from_numpy(d_losses).to(DEV)
        check_backward(x, dtype, ids, renormalize, moe.moe_router_backward(xd, tr, dw, dl), d_w, d_losses, counts, n)
        check_backward(x, dtype, ids, renormalize, moe.moe_router_backward(xd, r, dw), d_w, None, None, None)
        check_backward(x, dtype, ids, renormalize, moe.moe_router_backward(xd, tr, None, dl), None, d_losses, counts, n)
    assert not moe.moe_router_backward(xd, tr).any()  # no gradient in, none out


def test_router_gradient_is_the_difference_of_the_losses():
    """The logits' gradient against differences of the kernels' own losses and weights."""
    say("[gpu] router differences")
    rng = np.random.default_rng(5)
    T, E, k = 24, 16, 4
    x = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(DEV)
    g = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).to(DEV)
    dl = torch.tensor([1.0, 0.5], device=DEV)

    def loss(v):
        r = moe.moe_router_topk_losses(v, k)
        return (r.losses.double() * dl).sum().item() + (r.routing_w.double() * g).sum().item(), r

    base, r = loss(x)
    d = moe.moe_router_backward(x, r, g, dl)
    for t, e in [(0, 3), (5, 0), (11, int(r.expert_ids[11, 0])), (23, int(r.expert_ids[23, 3]))]:
        h = 1e-2
        up, ru = loss(x + h * torch.nn.functional.one_hot(torch.tensor(t * E + e), T * E).reshape(T, E).to(DEV))
        dn, rd = loss(x - h * torch.nn.functional.one_hot(torch.tensor(t * E + e), T * E).reshape(T, E).to(DEV))
        if not (torch.equal(ru.expert_ids, rd.expert_ids)):
            continue  # the choice changed: the loss is not smooth there
        # third derivatives of these losses are below 8 times the gradients' size here: h^2 / 6 * 8, plus fp32's
        # rounding of the two losses (size below 32) over 2 h
        assert abs((up - dn) / (2 * h) - d[t, e].item()) < 8 * h * h / 6 * g.abs().max().item() + 32 * 64 * U / h


def test_router_not_finite():
    say("[gpu] router with NaN and infinities")
    nan, inf = float("nan"), float("inf")
    x = torch.zeros((4, 16), device=DEV)
    x[0, 3], x[1, 5], x[2, :] = nan, inf, nan
    x[3, 7] = 2.0
    for dt in (torch.float32, torch.bfloat16):
        v = x.to(dt)
        r = moe.moe_router_topk_losses(v, 2)
        assert r.expert_ids.tolist() == [[0, 1], [5, 0], [-1, -1], [7, 0]]
        assert r.routing_w[:2].isnan().all() and not r.routing_w[2].any() and r.routing_w[3].isfinite().all()
        assert r.lse[:3].isnan().all() and r.lse[3].isfinite()
        assert r.losses.isnan().all() and r.tokens.item() == 4
        d = moe.moe_router_backward(v, moe.moe_router_topk(v, 2), torch.ones((4, 2), device=DEV))
        assert d[3].isfinite().all() and d[:3].isnan().all()


def test_router_no_tokens_and_all_padding():
    say("[gpu] router without tokens")
    for T in (0, 3):
        x = torch.full((T, 12), -float("inf"), device=DEV)
        r = moe.moe_router_topk_losses(x, 4)
        assert r.losses.tolist() == [0.0, 0.0] and r.tokens.item() == 0
        assert not r.counts.any() and not r.prob_mean.any() and (r.expert_ids == -1).all() and not r.routing_w.any()
        d = moe.moe_router_backward(x, r, torch.ones((T, 4), device=DEV), torch.ones(2, device=DEV))
        assert d.shape == (T, 12) and not d.any()


def test_router_unaligned_rows():
    """Logits and gradient that start anywhere: rows of a view, one element past an aligned address."""
    say("[gpu] router on unaligned logits")
    for dt, E in ((torch.bfloat16, 64), (torch.float32, 100)):
        buf = torch.randn(9 * E + 1, device=DEV).to(dt)
        x, y = buf[1:].view(9, E), buf[1:].clone().view(9, E)
        a, b = moe.moe_router_topk_losses(x, 5), moe.moe_router_topk_losses(y, 5)
        for f in ("expert_ids", "routing_w", "lse", "counts", "prob_mean", "losses"):
            assert torch.equal(getattr(a, f), getattr(b, f))
        g = torch.randn((9, 5), device=DEV)
        out = torch.empty(9 * E + 1, dtype=dt, device=DEV)[1:].view(9, E)
        assert torch.equal(moe.moe_router_backward(x, a, g, torch.ones(2, device=DEV), d_logits=out),
                           moe.moe_router_backward(y, b, g, torch.ones(2, device=DEV)))


def test_router_many_tokens_repeat():
    """Many workgroups: the statistics against sums over the kernel's own outputs, and the same bits again."""
    say("[gpu] router 70001 tokens")
    T, E, k = 70001, 96, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn((T, E), generator=g, device=DEV)
    x[-7:] = -float("inf")
    a, b = moe.moe_router_topk_losses(x, k, renormalize=False), moe.moe_router_topk_losses(x, k, renormalize=False)
    for f in ("expert_ids", "routing_w", "lse", "counts", "prob_mean", "losses", "tokens"):
        assert torch.equal(getattr(a, f), getattr(b, f))
    assert a.tokens.item() == T - 7 and torch.equal(a.counts.long(), torch.bincount(a.expert_ids[:-7].reshape(-1), minlength=E))
    p = torch.softmax(x[:-7].double(), 1)
    P = p.mean(0)
    assert ((a.prob_mean - P).abs() <= P * (T / 256 + 300 + 220) * U).all()
    top, ids = torch.topk(p, k)
    assert torch.equal(ids.int(), a.expert_ids[:-7])  # no ties among fp32 normals in a row's top here
    assert ((a.routing_w[:-7] - top).abs() <= top * 60 * 2 * U).all()


def test_router_other_stream_and_graph():
    """On a stream of its own, and captured: every replay equals an eager call on the inputs of that moment."""
    say("[gpu] router graph")
    T, E, k = 700, 128, 8
    x = torch.randn((T, E), device=DEV).to(torch.bfloat16)
    g, dl = torch.randn((T, k), device=DEV), torch.tensor([0.01, 0.001], device=DEV)
    keep = moe.moe_router_topk_losses(x, k)
    out = dict(expert_ids=keep.expert_ids, routing_w=keep.routing_w, lse=keep.lse, counts=keep.counts, tokens=keep.tokens,
               prob_mean=keep.prob_mean, losses=keep.losses,
               workspace=torch.empty(moe.router_workspace_bytes(T, E), dtype=torch.uint8, device=DEV))
    d = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        r = moe.moe_router_topk_losses(x, k, **out)
        moe.moe_router_backward(x, r, g, dl, d_logits=d)
        with torch.cuda.graph(graph, stream=s):
            r = moe.moe_router_topk_losses(x, k, **out)
            moe.moe_router_backward(x, r, g, dl, d_logits=d)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(3):
        x.copy_(torch.randn((T, E), device=DEV))
        ref = moe.moe_router_topk_losses(x, k)
        rd = moe.moe_router_backward(x, ref, g, dl)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for f in ("expert_ids", "routing_w", "lse", "counts", "tokens", "prob_mean", "losses"):
            assert torch.equal(getattr(ref, f), getattr(r, f)), (rep, f)
        assert torch.equal(rd, d)


def test_router_refusals():
    x = torch.zeros((4, 16), device=DEV)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x, 17)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x, 0)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x.t(), 2)
    with pytest.raises(TypeError):
        moe.moe_router_topk(x.half(), 2)
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_router_topk_losses(x, 2, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    r = moe.moe_router_topk(x, 2)
    with pytest.raises(ValueError):
        moe.moe_router_backward(x, r, None, torch.ones(2, device=DEV))  # no counts
    with pytest.raises(TypeError):
        moe.moe_router_backward(x, r, torch.ones((4, 2), dtype=torch.bfloat16, device=DEV))


def test_router_with_the_expert_step():
    """Router, expert step, its backward and the router's: one training pass as a layer runs it."""
    import oracle
    from gpu_util import bits, to_dev_bf16
    from workloads import make_random

    T, k, E, d, h = 300, 4, 12, 136, 72
    wl = make_random(T=T, k=k, E=E, d=d, h=h, seed=9)
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32))
    x[-20:] = -np.inf  # padding: no expert, a zero output row, no gradient
    x[:, 3] = -np.inf  # an expert that nobody may choose
    say(f"[gpu] router and expert step T={T} E={E}")
    xd = x.to(DEV)
    X, w_ug, w_down = to_dev_bf16(wl.x), to_dev_bf16(wl.w_ug), to_dev_bf16(wl.w_down)
    r = moe.moe_router_topk_losses(xd, k)
    y, _, h_buf, y_perm = moe.moe_expert_forward(X, r.expert_ids, r.routing_w, w_ug, w_down)
    p = moe.moe_permute(X, r.expert_ids, E)
    dy = torch.from_numpy(rng.normal(size=(T, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    grads = moe.moe_expert_backward(dy, p, r.routing_w, w_ug, w_down, h_buf, y_perm)
    dl = torch.tensor([0.01, 0.001], device=DEV)
    d_x = moe.moe_router_backward(xd, r, grads["d_routing_w"], dl)
    torch.cuda.synchronize()
    ids, w, lse = orr.topk(x.double().numpy(), k, True)
    np.testing.assert_array_equal(r.expert_ids.cpu().numpy(), ids)
    assert torch.equal(p.counts, r.counts) and r.counts[3].item() == 0
    ref = oracle.moe_expert_forward(wl.x, ids, w.astype(np.float32), wl.w_ug, wl.w_down)
    from parity import compare_bf16
    compare_bf16(bits(y), ref.y, "y")
    assert not y[-20:].any() and not d_x[-20:].any()
    counts, n, _, _ = orr.losses(x.double().numpy(), ids)
    check_backward(x, "f32", ids, True, d_x, grads["d_routing_w"].cpu().numpy(), dl.cpu().numpy().astype(np.float64), counts, n)
