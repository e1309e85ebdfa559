"""Norms before and after a block on the GPU against the 64-bit reference.

Tolerances: half a step of the output's type (bf16 2^-8, fp32 2^-24 of the value) and fp32 arithmetic, counted in 2^-24 of
the magnitudes of the terms: 40 for the values (sums of squares are 8 or 16 additions a lane, 10 between lanes and waves,
and enter through a square root; a dozen roundings and a 1-ulp reciprocal root), 100 for the gradients, which multiply
two such sums, and T + 100 for column sums over T rows.
"""

import itertools

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from oracle import norm as on

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, mag, terms, name):
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(f64(got) - want)
    tol = half * np.abs(want) + (1 + half) * terms * U * mag + 1e-38
    assert (err <= tol).all(), f"{name}: {np.nanmax(err / tol):.3g} times its tolerance"


def inputs(T, d, stream, weights, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, sigma=1.0, mean=0.0):
        return (mean + sigma * torch.randn(shape, generator=g, device="cuda")).to(dtype)

    v = dict(r=normal((T, d), stream), y=normal((T, d), BF16, 0.4), w_post=normal((d,), weights, 0.3, 1.0),
             w_next=normal((d,), weights, 0.3, 1.0), dr=normal((T, d), stream), dn=normal((T, d), BF16),
             dn2=normal((T, d), BF16))
    v["gate"] = {"none": None, "token": normal((T, 1), F32), "channel": normal((d,), weights)}[gate]
    return v


def check(T, d, stream, weights, post, gate, nxt, a=0.75, b=1.5, eps=1e-5, seed=0):
    v = inputs(T, d, stream, weights, gate, seed)
    kw = dict(post_norm=post, w_post=v["w_post"] if post else None, gate=v["gate"], residual_scale=a, branch_scale=b,
              next_norm=nxt, w_next=v["w_next"] if nxt else None, eps=eps)
    x, n = moe.moe_residual_norm(v["y"], v["r"], **kw)
    okw = dict(post=post, w_post=f64(v["w_post"]), gate=1.0 if gate == "none" else f64(v["gate"]), a=a, b=b, nxt=nxt,
               w_next=f64(v["w_next"]), eps=eps)
    rx, rn, mx, mn = on.forward(f64(v["r"]), f64(v["y"]), **okw)
    assert x.dtype == stream
    close(x, rx, mx, 40, "r'")
    if nxt:
        close(n, rn, mn, 40, "n")
    else:
        assert n is None
    for dr, more in ((v["dr"], None), (None, v["dn2"])) if nxt else ((v["dr"], None),):
        g = moe.moe_residual_norm_backward(dr, v["dn"] if nxt else None, v["y"], x, d_n_add=more, **kw)
        dn = None if not nxt else f64(v["dn"]) + (0 if more is None else f64(more))
        ref = on.backward(f64(dr), dn, f64(x), f64(v["y"]), gate_kind=gate, **okw)
        got = dict(r=g.d_r, y=g.d_y, gate=g.d_gate, w_post=g.d_w_post, w_next=g.d_w_next)
        assert {k for k, t in got.items() if t is not None} == set(ref)
        for k, (want, mag) in ref.items():
            terms = 100 + (T if k in ("w_post", "w_next") or (k == "gate" and gate == "channel") else 0)
            terms += d // 8 if k == "gate" and gate == "token" else 0
            assert got[k].dtype == {"r": stream, "y": BF16}.get(k, F32)
            close(got[k], want, mag, terms, f"gradient of {k}")


@pytest.mark.parametrize("post,gate,nxt", list(itertools.product((False, True), ("none", "token", "channel"), (False, True))))
@pytest.mark.parametrize("stream,weights", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_forms(post, gate, nxt, stream, weights):
    check(7, 136, stream, weights, post, gate, nxt)


@pytest.mark.parametrize("T,d", [(1, 8), (2, 16), (65, 24), (3, 504), (5, 512), (5, 520), (4, 2048), (33, 2056),
                                 (3, 2880), (2, 8192), (3, 8200), (2, 16376), (2, 16384), (1100, 64),
                                 (3, 120), (5, 128), (67, 136), (2, 248), (7, 256), (35, 264), (20001, 72), (9001, 200),
                                 (5, 10912), (3, 12288)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_sizes(T, d, stream):
    if d <= 4096:  # (the reference's Jacobian is a matrix of d x d)
        check(T, d, stream, F32, True, "channel", True)
        check(T, d, stream, BF16, False, "token", True)
    else:
        check(T, d, stream, BF16, True, "token", True)


@pytest.mark.parametrize("T,d", [(1, 8), (4, 512), (9, 1000), (2, 9000), (1000, 40)])
@pytest.mark.parametrize("stream,weight", [(BF16, BF16), (F32, F32), (BF16, None)])
def test_before(T, d, stream, weight):
    v = inputs(T, d, stream, weight or F32, "none", 5)
    w = None if weight is None else v["w_next"]
    n = moe.moe_rmsnorm(v["r"], w, eps=1e-4)
    rw = 1.0 if w is None else f64(w)
    _, rn, _, mn = on.forward(f64(v["r"]), w_next=rw, eps=1e-4)
    close(n, rn, mn, 40, "n")
    for add, more in ((v["dr"], v["dn2"]), (None, None)):
        dx, dw = moe.moe_rmsnorm_backward(v["dn"], v["r"], w, eps=1e-4, dx_add=add, dy_add=more)
        dn = f64(v["dn"]) + (0 if more is None else f64(more))
        ref = on.backward(f64(add), dn, f64(v["r"]), w_next=rw, eps=1e-4)
        close(dx, *ref["r"], 100, "dx")
        if w is None:
            assert dw is None
        else:
            close(dw, *ref["w_next"], T + 100, "dw")


def test_rows_of_zeros_and_scales():
    """A zero row normalises to zeros; tiny and huge rows keep their direction."""
    r = torch.zeros((4, 64), device="cuda")
    r[1], r[2], r[3] = 1e-15, 1e15, 3.0
    n = moe.moe_rmsnorm(r, None, eps=1e-6)
    assert not n[0].any() and torch.isfinite(n).all()
    close(n, on.forward(f64(r), eps=1e-6)[1], np.abs(on.forward(f64(r), eps=1e-6)[1]), 40, "n")
    dn = torch.randn((4, 64), device="cuda").to(BF16)
    dx, _ = moe.moe_rmsnorm_backward(dn, r, None, eps=1e-6)
    close(dx, *on.backward(None, f64(dn), f64(r), eps=1e-6)["r"], 100, "dx")


def test_what_is_not_finite_stays_in_its_row():
    v = inputs(6, 200, BF16, F32, "token", 2)
    v["y"][2, 7], v["r"][4, 9] = float("nan"), float("inf")
    x, n = moe.moe_residual_norm(v["y"], v["r"], post_norm=True, gate=v["gate"], w_next=v["w_next"])
    bad = ~torch.isfinite(n).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]
    clean = inputs(6, 200, BF16, F32, "token", 2)
    x2, n2 = moe.moe_residual_norm(clean["y"], clean["r"], post_norm=True, gate=v["gate"], w_next=v["w_next"])
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    assert torch.equal(x[keep], x2[keep]) and torch.equal(n[keep], n2[keep])


def test_no_rows():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    gate = torch.ones(64, device="cuda")
    x, n = moe.moe_residual_norm(e, e, post_norm=True, w_post=w, gate=gate, w_next=w)
    assert x.shape == n.shape == (0, 64)
    g = moe.moe_residual_norm_backward(e, e, e, e, post_norm=True, w_post=w, gate=gate, w_next=w)
    for t in (g.d_w_post, g.d_w_next, g.d_gate):
        assert t.shape == (64,) and not t.any()  # sums over no rows


@pytest.mark.parametrize("stream", [BF16, F32])
def test_in_place_and_repeatable(stream):
    v = inputs(300, 1032, stream, BF16, "channel", 3)
    kw = dict(post_norm=True, w_post=v["w_post"], gate=v["gate"], residual_scale=0.5, w_next=v["w_next"])
    x, n = moe.moe_residual_norm(v["y"], v["r"], **kw)
    g = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, **kw)
    for _ in range(3):
        again = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, **kw)
        assert all(torch.equal(getattr(g, f), getattr(again, f)) for f in ("d_r", "d_y", "d_gate", "d_w_post", "d_w_next"))
    r, dr, dn = v["r"].clone(), v["dr"].clone(), v["dn"].clone()
    x2, n2 = moe.moe_residual_norm(v["y"], r, r_out=r, **kw)
    assert x2.data_ptr() == r.data_ptr() and torch.equal(x, x2) and torch.equal(n, n2)
    g2 = moe.moe_residual_norm_backward(dr, dn, v["y"], x, d_r=dr, d_y=dn, **kw)
    assert torch.equal(g2.d_r, g.d_r) and torch.equal(g2.d_y, g.d_y) and g2.d_r.data_ptr() == dr.data_ptr()


@pytest.mark.parametrize("T,d,kind", [(70, 64, "token"), (70, 200, "token"), (40, 2880, "token"), (9, 8200, "token"),
                                      (33, 1032, "channel")])
def test_every_gradient_over_an_input(T, d, kind):
    v = inputs(T, d, F32, F32, kind, 12)
    kw = dict(post_norm=True, w_post=v["w_post"], w_next=v["w_next"])
    x, _ = moe.moe_residual_norm(v["y"], v["r"], gate=v["gate"], **kw)
    want = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, gate=v["gate"], **kw)
    got = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, gate=v["gate"], d_r=x, d_y=v["y"], d_gate=v["gate"],
                                         **kw)
    assert got.d_gate.data_ptr() == v["gate"].data_ptr() and got.d_r.data_ptr() == x.data_ptr()
    for f in ("d_r", "d_y", "d_gate", "d_w_post", "d_w_next"):
        assert torch.equal(getattr(got, f), getattr(want, f)), f


def test_gradient_against_differences():
    """Two points along a random direction, in fp32 where the stream allows it: the difference quotient of the sum the
    gradients belong to agrees to the rounding of n to bf16, averaged over T d values, and the step's third order."""
    T, d = 64, 256
    v = inputs(T, d, F32, F32, "channel", 4)
    kw = dict(post_norm=True, branch_scale=0.5)
    names = ("w_post", "gate", "w_next")

    def total(p):
        x, n = moe.moe_residual_norm(v["y"], p["r"], w_post=p["w_post"], gate=p["gate"], w_next=p["w_next"], **kw)
        return float((x.double() * v["dr"].double()).sum() + (n.double() * v["dn"].double()).sum()), x

    base = {k: v[k] for k in ("r",) + names}
    _, x = total(base)
    g = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, w_post=v["w_post"], gate=v["gate"],
                                       w_next=v["w_next"], **kw)
    grads = dict(r=g.d_r, w_post=g.d_w_post, gate=g.d_gate, w_next=g.d_w_next)
    h = 2.0 ** -5
    gen = torch.Generator(device="cuda").manual_seed(9)
    for k in grads:
        e = torch.randn(base[k].shape, generator=gen, device="cuda")
        up, down = total({**base, k: base[k] + h * e})[0], total({**base, k: base[k] - h * e})[0]
        want = float((grads[k].double() * e.double()).sum())
        # n's roundings: at most 2^-8 |n| each, |n| about 1.1, independent: T d of them add up to sqrt(T d) 2^-8, twice,
        # over 2 h, six deviations of it; the third order: h^2 times a bounded form of the same size as `want`'s scale
        scale = float(grads[k].double().norm() * e.double().norm()) / np.sqrt(e.numel())
        tol = 6 * np.sqrt(T * d) * 2.0 ** -8 / h + 8 * h * h * scale * 6
        assert abs((up - down) / (2 * h) - want) < tol, k


def test_streams_and_a_graph():
    v = inputs(64, 512, BF16, BF16, "channel", 6)
    kw = dict(post_norm=True, w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"])

    def step(ws):
        x, n = moe.moe_residual_norm(v["y"], v["r"], **kw)
        g = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, workspace=ws, **kw)
        return [x, n, g.d_r, g.d_y, g.d_gate, g.d_w_post, g.d_w_next]

    spaces = [torch.empty(moe.norm_workspace_bytes(64, 512), dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step(spaces[0])
    want = step(spaces[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on_side, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(spaces[0])
    for seed in (6, 7, 8):
        fresh = inputs(64, 512, BF16, BF16, "channel", seed)
        for k in ("r", "y", "dr", "dn"):
            v[k].copy_(fresh[k])
        graph.replay()
        want = step(spaces[1])  # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_refusals():
    v = inputs(4, 64, BF16, F32, "none")
    x, w = v["r"], v["w_next"]
    for call in (lambda: moe.moe_rmsnorm(x.t(), w), lambda: moe.moe_rmsnorm(x[:, ::2], w[:32].contiguous()),
                 lambda: moe.moe_rmsnorm(x, w[:32].contiguous()), lambda: moe.moe_rmsnorm(x, w.cpu()),
                 lambda: moe.moe_residual_norm(x[:2], x), lambda: moe.moe_residual_norm(x, x, w_post=w),
                 lambda: moe.moe_residual_norm(x, x, next_norm=False, w_next=w),
                 lambda: moe.moe_residual_norm(x, x, gate=torch.ones((2, 1), device="cuda")),
                 lambda: moe.moe_residual_norm_backward(None, None, x, x, next_norm=False),
                 lambda: moe.moe_residual_norm_backward(x, x, x, x, next_norm=False),
                 lambda: moe.moe_rmsnorm_backward(x, x, w, workspace=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_rmsnorm(x.half(), w), lambda: moe.moe_rmsnorm(x, w.half()),
                 lambda: moe.moe_residual_norm(x.float(), x), lambda: moe.moe_residual_norm(x, x, w_next=w, post_norm=True,
                                                                                             w_post=w.to(BF16)),
                 lambda: moe.moe_residual_norm(x, x, gate=torch.ones((4, 1), dtype=BF16, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm(torch.zeros((2, 12), device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(moe.MoeError):
        moe.moe_rmsnorm_backward(x, x, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
