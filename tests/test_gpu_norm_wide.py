"""Wide rows on the GPU with a gate per channel against 64 bits: two and three column sums, weights that lie in LDS and
weights that do not fit it (three sums of more than 10240 columns).

Tolerances as for narrower rows, in 2^-24 of the magnitudes of the terms: 40 for the values, 100 for the gradients and T
more for column sums over T rows (two vectors a lane make the lane's part of a row's sum 16 additions, counted there).
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from oracle import norm as on
from test_gpu_norm import close, f64, inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def check(T, d, stream, weights, post, nxt, dr_too, more_too, seed, a=0.75, b=1.5, eps=1e-5):
    v = inputs(T, d, stream, weights, "channel", seed)
    kw = dict(post_norm=post, w_post=v["w_post"] if post else None, gate=v["gate"], residual_scale=a, branch_scale=b,
              next_norm=nxt, w_next=v["w_next"] if nxt else None, eps=eps)
    okw = dict(post=post, w_post=f64(v["w_post"]), gate=f64(v["gate"]), a=a, b=b, nxt=nxt, w_next=f64(v["w_next"]), eps=eps)
    x, n = moe.moe_residual_norm(v["y"], v["r"], **kw)
    rx, rn, mx, mn = on.forward(f64(v["r"]), f64(v["y"]), **okw)
    close(x, rx, mx, 40, "r'")
    if nxt:
        close(n, rn, mn, 40, "n")
    dr, more = v["dr"] if dr_too else None, v["dn2"] if more_too else None
    g = moe.moe_residual_norm_backward(dr, v["dn"] if nxt else None, v["y"], x, d_n_add=more, **kw)
    dn = f64(v["dn"]) + (0 if more is None else f64(more))
    ref = on.backward(f64(dr), dn, f64(x), f64(v["y"]), gate_kind="channel", through=on.through_wide_norm, **okw)
    got = dict(r=g.d_r, y=g.d_y, gate=g.d_gate, w_post=g.d_w_post, w_next=g.d_w_next)
    assert {k for k, t in got.items() if t is not None} == set(ref)
    for k, (want, mag) in ref.items():
        assert got[k].dtype == {"r": stream, "y": BF16}.get(k, F32)
        close(got[k], want, mag, 100 + (0 if k in ("r", "y") else T), f"gradient of {k}")


# a row to a workgroup from 4104 columns on; 256 of them, so 300 rows are two turns
@pytest.mark.parametrize("T,d", [(3, 4104), (300, 5120), (2, 8192), (3, 8200), (2, 10240), (3, 10248), (2, 10920),
                                 (300, 11264), (2, 16376), (3, 16384)])
@pytest.mark.parametrize("stream,weights", [(BF16, BF16), (F32, BF16), (F32, F32)])
def test_three_column_sums(T, d, stream, weights):
    check(T, d, stream, weights, True, True, True, False, 1)
    check(T, d, stream, weights, True, True, False, True, 2)


@pytest.mark.parametrize("d", [4104, 8200, 16384])
@pytest.mark.parametrize("post,nxt", [(False, True), (True, False)])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_two_column_sums(d, post, nxt, stream):
    check(5, d, stream, BF16, post, nxt, True, nxt, 3)


@pytest.mark.parametrize("d", [5120, 10248, 16384])
def test_wide_rows_repeat_and_go_in_place(d):
    v = inputs(280, d, F32, F32, "channel", 4)
    kw = dict(post_norm=True, w_post=v["w_post"], gate=v["gate"], w_next=v["w_next"])
    x, _ = moe.moe_residual_norm(v["y"], v["r"], **kw)
    names = ("d_r", "d_y", "d_gate", "d_w_post", "d_w_next")
    want = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, **kw)
    for _ in range(2):
        again = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, **kw)
        assert all(torch.equal(getattr(want, f), getattr(again, f)) for f in names)
    # every gradient over an input of its type and shape, the weights' too
    got = moe.moe_residual_norm_backward(v["dr"], v["dn"], v["y"], x, d_r=x, d_y=v["y"], d_gate=v["gate"],
                                         d_w_post=v["w_post"], d_w_next=v["w_next"], **kw)
    assert all(torch.equal(getattr(want, f), getattr(got, f)) for f in names)
    assert got.d_w_next.data_ptr() == v["w_next"].data_ptr() and got.d_r.data_ptr() == x.data_ptr()
    assert np.isfinite(f64(got.d_gate)).all()
