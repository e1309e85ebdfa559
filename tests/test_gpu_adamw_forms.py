"""Forms of the AdamW step on the GPU that small tests of others do not reach: 32-bit moments with bf16 parameters rounded
at random, and 8-bit moments with an eps below 1e-12, whose step takes the exact root and quotient.

Tolerances in fp32 steps of 2^-24 as for the other forms: 3 of |p| and 12 of the update's size, from the moments that the
reference gives to the bit.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from oracle import adamw as oa
from test_gpu_adamw import BF16, F32, HYPER, ORACLE, SIZES, U, f32, f64, padded, place, rounded, tensors

pytestmark = pytest.mark.gpu


def carried(values, low):
    """bf16 values (as fp32) of fp32 ones whose dropped half has 16 random bits added."""
    i = values.view(np.uint32).astype(np.int64) + low
    return ((i >> 16) << 16).astype(np.uint32).view(np.float32)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("grad", [BF16, F32])
@pytest.mark.parametrize("seed", [0, 77])
def test_32_bit_moments_with_parameters_rounded_at_random(seed, grad, offset):
    """Against fp32 parameters of the same values: the same moments to the bit, and each parameter what its place's random
    half makes of the fp32 result; those against 64 bits."""
    params = tensors(SIZES + [300000], (BF16, F32), 31, offset=offset)
    state = moe.moe_adamw_state(params)
    wide = [p.float().clone() for p in params]
    other = moe.moe_adamw_state(wide)
    for t in (1, 2, 9):
        grads = tensors(SIZES + [300000], (grad,), 40 + t, 1e-2, offset)
        for w, p in zip(wide, params):
            w.copy_(p)
        before = [(f64(p), f64(state.exp_avg[place(state, i)]), f64(state.exp_avg_sq[place(state, i)]))
                  for i, p in enumerate(params)]
        moe.moe_adamw_step(state, grads, step=t, seed=seed, **HYPER)
        moe.moe_adamw_step(other, grads, step=t, **HYPER)
        assert torch.equal(state.exp_avg, other.exp_avg) and torch.equal(state.exp_avg_sq, other.exp_avg_sq)
        low = oa.random_bits(seed, t, np.arange(state.len)) & 0xFFFF
        for i, (p, w) in enumerate(zip(params, wide)):
            at = place(state, i)
            p0, m0, v0 = before[i]
            p1, m1, v1, update = oa.step64(p0, f64(grads[i]), m0, v0, t=t, **ORACLE)
            mag_m = np.abs(0.9 * m0) + np.abs(0.1 * f64(grads[i]))
            slope = np.abs(update) / np.maximum(np.abs(m1), 1e-300) * mag_m
            rounded(w, p1, 3 * np.abs(p0) + 20 * np.abs(update) + 8 * slope)
            want = f32(w) if p.dtype == F32 else carried(f32(w), low[at])
            np.testing.assert_array_equal(f32(p), want)


def test_large_tensors_rounded_at_random():
    """Enough values for two passes a chunk, an end inside a chunk, a tensor that begins off a vector."""
    sizes = [9_000_003, 40_001]
    params = tensors(sizes, (BF16,), 32, offset=1)
    params[0] = params[0].clone()  # (aligned)
    wide = [p.float().clone() for p in params]
    grads = tensors(sizes, (BF16,), 33, 1e-2)
    state, other = moe.moe_adamw_state(params), moe.moe_adamw_state(wide)
    moe.moe_adamw_step(state, grads, step=4, seed=123456789, **HYPER)
    moe.moe_adamw_step(other, grads, step=4, **HYPER)
    assert torch.equal(state.exp_avg, other.exp_avg) and torch.equal(state.exp_avg_sq, other.exp_avg_sq)
    for i, (p, w) in enumerate(zip(params, wide)):
        low = oa.random_bits(123456789, 4, np.arange(state.places[i], state.places[i] + sizes[i])) & 0xFFFF
        np.testing.assert_array_equal(f32(p), carried(f32(w), low))


def test_random_parameters_that_are_not_finite():
    """What is not finite rounds as usual: an infinity stays one, a NaN does not turn into an infinity."""
    p = [torch.full((4100,), 1.0, dtype=BF16, device="cuda")]
    p[0][5], p[0][4099] = float("inf"), float("-inf")
    g = torch.zeros(4100, device="cuda")
    g[2000] = float("nan")
    state = moe.moe_adamw_state(p)
    moe.moe_adamw_step(state, [g], step=1, seed=5, **HYPER)
    assert p[0][5] == float("inf") and p[0][4099] == float("-inf") and torch.isnan(p[0][2000])
    p[0][[5, 2000, 4099]] = 1.0
    assert torch.isfinite(p[0]).all() and (p[0] != 1).any()


@pytest.mark.parametrize("eps", [1e-20, 1e-13])
@pytest.mark.parametrize("seed", [None, 6])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("p", [(BF16,), (F32, BF16)])
def test_8_bit_moments_with_a_small_eps(p, master, seed, eps):
    params = tensors(SIZES, p, 51)
    state = moe.moe_adamw_state(params, bits=8, master=master)
    mq, ms = np.zeros(state.len, np.uint8), np.zeros(state.len // 32, np.uint8)
    vq, vs = mq.copy(), ms.copy()
    for t in (1, 2):
        grads = tensors(SIZES, (F32,), 60 + t, 1e-2)
        # second moments below 2^-126, which the shorter step takes for 0
        grads[9][:4000] *= 1e-18
        grads[9][64:96] = 0
        old = [f32(state.master[place(state, i)] if master else q) for i, q in enumerate(params)]
        moe.moe_adamw_step(state, grads, step=t, seed=seed, **{**HYPER, "eps": eps})
        m, v = oa.of_e4m3(mq, ms).astype(np.float32), oa.of_e5m3(vq, vs).astype(np.float32)
        m, v = oa.moments32(padded(state, [f32(d) for d in grads]), m, v, 0.9, 0.999)
        bits = None if seed is None else oa.random_bits(seed, t, np.arange(state.len))
        mq, ms = oa.to_e4m3(m)
        vq, vs = oa.to_e5m3(v, None if bits is None else bits >> 16)
        for got, want in ((state.exp_avg.q, mq), (state.exp_avg.scales, ms), (state.exp_avg_sq.q, vq),
                          (state.exp_avg_sq.scales, vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        for i, q in enumerate(params):
            at = place(state, i)
            m1, v1, p0 = m[at].astype(float), v[at].astype(float), old[i].astype(float)
            update = 3e-3 / (1 - 0.9 ** t) * m1 / (np.sqrt(v1 / (1 - 0.999 ** t)) + eps)
            want, mag = (1 - 3e-3 * 0.1) * p0 - update, 3 * np.abs(p0) + 12 * np.abs(update)
            if master:
                rounded(state.master[at], want, mag)
                assert torch.equal(q, state.master[at].to(q.dtype))
            elif seed is None or q.dtype == F32:
                rounded(q, want, mag)
            else:  # one of the two neighbours
                err = np.abs(f64(q) - want)
                assert (err <= torch.finfo(BF16).eps * np.abs(want) + 2 * U * mag + 1e-40).all()


def test_parameters_that_changed_type_or_order_in_memory():
    """Refused on the GPU as on the host, and nothing is written."""
    memory = torch.ones(128, device="cuda")
    square = torch.nn.Parameter(torch.arange(36.0, device="cuda").reshape(6, 6))
    state = moe.moe_adamw_state([memory[:64], square])
    grads = [torch.ones(64, device="cuda"), torch.ones((6, 6), device="cuda")]
    state.params[0] = memory.view(BF16)[:64]
    with pytest.raises(TypeError):
        moe.moe_adamw_step(state, grads, lr=1e-3)
    state.params[0] = memory[:64]
    square.data = square.data.t()
    with pytest.raises(ValueError):
        moe.moe_adamw_step(state, grads, lr=1e-3)
    square.data = square.data.t()
    state.exp_avg_sq = state.exp_avg
    with pytest.raises(ValueError):
        moe.moe_adamw_step(state, grads, lr=1e-3)
    assert (memory == 1).all() and torch.equal(square.data, torch.arange(36.0, device="cuda").reshape(6, 6))
    state.exp_avg_sq = torch.zeros_like(state.exp_avg)
    moe.moe_adamw_step(state, grads, lr=1e-3)
    assert (memory[:64] != 1).all() and (memory[64:] == 1).all()
