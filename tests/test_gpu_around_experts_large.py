"""Norms, AdamW and 4-bit experts past 2^31 elements: rows and values behind the border come out as alone."""

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_norm_rows():
    T, d = 270_000, 8192  # 2.2 G values
    w = torch.rand(d, device="cuda") + 0.5
    r = torch.empty((T, d), dtype=BF16, device="cuda")
    row = torch.randn((7, d), device="cuda").to(BF16)
    for lo in range(0, T, 50_000):
        r[lo:lo + 50_000] = row[0]
    r[-7:] = row
    n = moe.moe_rmsnorm(r, w)
    assert torch.equal(n[-7:], moe.moe_rmsnorm(row, w)) and torch.equal(n[1], n[T - 100])
    x, n = moe.moe_residual_norm(n, r, post_norm=True, w_post=w, gate=w, w_next=w, r_out=r)
    y = moe.moe_rmsnorm(row, w)
    x7, n7 = moe.moe_residual_norm(y, row, post_norm=True, w_post=w, gate=w, w_next=w)
    assert torch.equal(x[-7:], x7) and torch.equal(n[-7:], n7)
    # gradients of rows do not depend on the others'; n serves as its own gradient
    y = torch.empty_like(n).copy_(n)
    g = moe.moe_residual_norm_backward(x, n, y, x, post_norm=True, w_post=w, gate=w, w_next=w, d_r=x, d_y=y)
    g7 = moe.moe_residual_norm_backward(x7, n7, n7, x7, post_norm=True, w_post=w, gate=w, w_next=w)
    assert torch.equal(g.d_r[-7:], g7.d_r) and torch.equal(g.d_y[-7:], g7.d_y)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_values(bits):
    n = (1 << 31) + 4133
    p = [torch.zeros(64, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")]
    g = [torch.full((64,), 0.5, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")]
    tail = torch.randn(4133 + 512, device="cuda").to(BF16)
    g[1][-tail.numel():] = tail
    state = moe.moe_adamw_state(p, bits=bits)
    moe.moe_adamw_step(state, g, lr=1e-2, step=2)
    alone = [torch.zeros_like(tail)]
    one = moe.moe_adamw_state(alone, bits=bits)
    moe.moe_adamw_step(one, [tail], lr=1e-2, step=2)
    assert torch.equal(p[1][-tail.numel():], alone[0]) and not p[1][:1 << 20].any()
    first = state.places[1] + n - tail.numel()
    if bits == 32:
        assert torch.equal(state.exp_avg[first:first + tail.numel()], one.exp_avg[:tail.numel()])
    else:
        assert torch.equal(state.exp_avg.q[first:first + tail.numel()], one.exp_avg.q[:tail.numel()])
        assert torch.equal(state.exp_avg_sq.q[first:first + tail.numel()], one.exp_avg_sq.q[:tail.numel()])


def test_int4_weights():
    E, K, N = 160, 4096, 16384  # 5.4 GB of packed weights
    q = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((E, K // 128, N), 0.02, dtype=BF16, device="cuda")
    z = torch.randint(0, 16, (E, K // 128, N), dtype=torch.uint8, device="cuda")
    x = torch.randn((6, K), device="cuda").to(BF16)
    counts = [0] * E
    counts[0], counts[E - 1] = 2, 4
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_projection_int4(x, off, moe.Int4(q, s, z, K))
    for e, rows in ((0, slice(0, 2)), (E - 1, slice(2, 6))):
        one = moe.Int4(q[e:e + 1].contiguous(), s[e:e + 1].contiguous(), z[e:e + 1].contiguous(), K)
        own = torch.tensor([0, rows.stop - rows.start], dtype=torch.int32, device="cuda")
        assert torch.equal(y[rows], moe.moe_grouped_projection_int4(x[rows].contiguous(), own, one))
    back = moe.moe_int4_dequantize_weights(moe.Int4(q[-1:].contiguous(), s[-1:].contiguous(), z[-1:].contiguous(), K))
    want = x[2:].double() @ back[0].double().T
    # the weights read back are rounded to bf16 once, the result too
    assert float((y[2:].double() - want).norm() / want.norm()) < 2 * 2.0 ** -8


def test_int4_token_rows():
    """Token rows of more than 2 GiB, read through the dispatch order, by both kinds of tiles."""
    T, d, h, E = 600_000, 2048, 32, 4
    x = torch.zeros((T, d), dtype=BF16, device="cuda")
    tail = torch.randn((40, d), device="cuda").to(BF16)
    x[-40:] = tail
    w = moe.moe_int4_quantize_weights(torch.randn((E, 2 * h, d), device="cuda").to(BF16), "out_in", group=32)
    perm = torch.zeros(T, dtype=torch.int32, device="cuda")
    perm[:40] = torch.arange(T - 40, T, device="cuda")
    off = torch.tensor([0, 1, 1, 20, 40], dtype=torch.int32, device="cuda")
    got = moe.moe_gemm_up_swiglu_int4(x, off, w, perm=perm, k=1)[:40]
    want = moe.moe_gemm_up_swiglu_int4(tail, off, w)
    # other tiles add in another order: both round once from sums within 2^-16 of each other, one step of bf16 apart at most
    near = (got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -14 * want.double().abs().max()
    assert near.all()
