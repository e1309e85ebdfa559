"""AdamW over many tensors on the GPU: fp32 results against 64 bits, 8-bit moments bit for bit.

Tolerances in fp32 steps of 2^-24: m = m b1 + g (1 - b1) has two products, two constants and a sum (5 of the terms'
magnitudes), v one more product; the update's quotient, root, constants and products make 12 of its size on top of
what m's and half of v's relative errors carry over (8), and p is multiplied and subtracted (3 of |p|).
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from oracle import adamw as oa

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
ORACLE = dict(lr=3e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def f32(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def tensors(sizes, dtypes, seed=0, sigma=0.02, offset=0):
    """One tensor a size; `offset` values into their memory."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.randn(n + offset, generator=g, device="cuda") * sigma).to(dtypes[i % len(dtypes)])
        out.append(t[offset:])
    return out


def rounded(got, want, mag):
    """Within half a step of the output's type and `mag` fp32 roundings."""
    half = torch.finfo(got.dtype).eps / 2
    err, tol = np.abs(f64(got) - want), half * np.abs(want) + (1 + half) * U * mag + 1e-45
    assert (err <= tol).all(), f"{(err / tol).max():.3g} times its tolerance"


def place(state, i):
    return slice(state.places[i], state.places[i] + state.params[i].numel())


SIZES = [1, 7, 8, 31, 32, 33, 4095, 4096, 4097, 10000, 0, 5]


@pytest.mark.parametrize("p,g", [((F32,), (F32,)), ((BF16,), (BF16,)), ((BF16, F32), (F32, BF16, BF16))])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps_in_32_bits(p, g, master, offset):
    params = tensors(SIZES, p, 1, offset=offset)
    state = moe.moe_adamw_state(params, master=master)
    for t in (1, 2, 3):
        grads = tensors(SIZES, g, 10 + t, 1e-2, offset)
        before = [(f64(state.master[place(state, i)] if master else q), f64(state.exp_avg[place(state, i)]),
                   f64(state.exp_avg_sq[place(state, i)])) for i, q in enumerate(params)]
        moe.moe_adamw_step(state, grads, step=t, **HYPER)
        for i, (q, d) in enumerate(zip(params, grads)):
            p0, m0, v0 = before[i]
            p1, m1, v1, update = oa.step64(p0, f64(d), m0, v0, t=t, **ORACLE)
            mag_m = np.abs(0.9 * m0) + np.abs(0.1 * f64(d))
            rounded(state.exp_avg[place(state, i)], m1, 5 * mag_m)
            rounded(state.exp_avg_sq[place(state, i)], v1, 6 * v1)
            slope = np.abs(update) / np.maximum(np.abs(m1), 1e-300) * mag_m
            mag = 3 * np.abs(p0) + 20 * np.abs(update) + 8 * slope
            if master:
                rounded(state.master[place(state, i)], p1, mag)
                assert torch.equal(q, state.master[place(state, i)].to(q.dtype))
            else:
                rounded(q, p1, mag)
    used = torch.zeros(state.len, dtype=torch.bool, device="cuda")
    for i in range(len(params)):
        used[place(state, i)] = True
    assert not state.exp_avg[~used].any() and not state.exp_avg_sq[~used].any()
    if master:
        assert not state.master[~used].any()


def padded(state, values):
    out = np.zeros(state.len, np.float32)
    for i, v in enumerate(values):
        out[place(state, i)] = v
    return out


@pytest.mark.parametrize("seed", [None, 0, 4294967295])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("p,g", [((BF16,), (BF16,)), ((F32, BF16), (F32,))])
def test_moments_in_8_bits_to_the_bit(seed, master, p, g):
    params = tensors(SIZES, p, 2)
    state = moe.moe_adamw_state(params, bits=8, master=master)
    mq, ms = np.zeros(state.len, np.uint8), np.zeros(state.len // 32, np.uint8)
    vq, vs = mq.copy(), ms.copy()
    for t in (1, 2, 3):
        grads = tensors(SIZES, g, 20 + t, 1e-2 * 30 ** t)
        grads[9][3:2000] *= 1e-6  # blocks of small values beside large ones
        grads[9][64:128] = 0
        old = [f32(state.master[place(state, i)] if master else q) for i, q in enumerate(params)]
        moe.moe_adamw_step(state, grads, step=t, seed=seed, **HYPER)
        m = oa.of_e4m3(mq, ms).astype(np.float32)
        v = oa.of_e5m3(vq, vs).astype(np.float32)
        m, v = oa.moments32(padded(state, [f32(d) for d in grads]), m, v, 0.9, 0.999)
        bits = None if seed is None else oa.random_bits(seed, t, np.arange(state.len))
        mq, ms = oa.to_e4m3(m)
        vq, vs = oa.to_e5m3(v, None if bits is None else bits >> 16)
        for got, want in ((state.exp_avg.q, mq), (state.exp_avg.scales, ms), (state.exp_avg_sq.q, vq),
                          (state.exp_avg_sq.scales, vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        # the step itself takes the moments before they are rounded
        for i, q in enumerate(params):
            at = place(state, i)
            m1, v1, p0 = m[at].astype(float), v[at].astype(float), old[i].astype(float)
            update = 3e-3 / (1 - 0.9 ** t) * m1 / (np.sqrt(v1 / (1 - 0.999 ** t)) + 1e-8)
            want, mag = (1 - 3e-3 * 0.1) * p0 - update, 3 * np.abs(p0) + 12 * np.abs(update)
            if master:
                rounded(state.master[at], want, mag)
            elif seed is None or q.dtype == F32:
                rounded(q, want, mag)
            else:  # one of the two neighbours
                err = np.abs(f64(q) - want)
                assert (err <= torch.finfo(BF16).eps * np.abs(want) + 2 * U * mag + 1e-40).all()
        got_m, got_v = moe.moe_adamw_moments(state)
        np.testing.assert_array_equal(f64(got_m), oa.of_e4m3(mq, ms))
        np.testing.assert_array_equal(f64(got_v), oa.of_e5m3(vq, vs))


def test_random_parameters_round_as_the_bits_say():
    """fp32 results against bf16 ones of the same step: the dropped half and the place's random half carry over."""
    n = 5000
    params = tensors([n], (BF16,), 3)
    copy = [params[0].float()]
    a, b = moe.moe_adamw_state(params, bits=8), moe.moe_adamw_state(copy, bits=8)
    grads = tensors([n], (F32,), 4)
    moe.moe_adamw_step(a, grads, step=5, seed=9, **HYPER)
    moe.moe_adamw_step(b, grads, step=5, seed=9, **HYPER)
    low = oa.random_bits(9, 5, np.arange(n)) & 0xFFFF
    i = f32(copy[0]).view(np.uint32).astype(np.int64) + low
    want = ((i >> 16) << 16).astype(np.uint32).view(np.float32)
    np.testing.assert_array_equal(f32(params[0]), want)


def test_a_small_second_moment_follows_its_gradients_on_average():
    """v is 1, g^2 is 1.5: the exact mean of 64 steps of 1 - 0.999 is 1.5 - 0.5 * 0.999^64. Rounded at random the mean over
    n values stays within six deviations: a step's rounding deviates by at most half a code, 1/16."""
    n, steps = 1 << 14, 64
    p = [torch.zeros(n, device="cuda")]
    state = moe.moe_adamw_state(p, bits=8)
    state.exp_avg_sq.q.fill_(240)
    state.exp_avg_sq.scales.fill_(97)
    assert (moe.moe_adamw_moments(state)[1] == 1).all()
    g = [torch.full((n,), 1.5 ** 0.5, device="cuda")]
    for t in range(1, steps + 1):
        moe.moe_adamw_step(state, g, step=t, seed=1, **HYPER)
    mean = float(moe.moe_adamw_moments(state)[1].double().mean())
    want = 1.5 - 0.5 * 0.999 ** steps
    assert abs(mean - want) < 6 * np.sqrt(steps / n) / 16 + steps * 2.0 ** -16 / 8 + steps * 2.0 ** -22
    still = moe.moe_adamw_state(p, bits=8)
    still.exp_avg_sq.q.fill_(240)
    still.exp_avg_sq.scales.fill_(97)
    moe.moe_adamw_step(still, g, step=1, **HYPER)
    assert (moe.moe_adamw_moments(still)[1] == 1).all()  # to nearest it does not move


def test_what_is_not_finite():
    n = 256
    for bits in (32, 8):
        params, grads = tensors([n], (F32,), 5), tensors([n], (F32,), 6)
        grads[0][40], grads[0][130] = float("nan"), float("inf")
        state = moe.moe_adamw_state(params, bits=bits)
        moe.moe_adamw_step(state, grads, step=1, **HYPER)
        bad = ~torch.isfinite(params[0])
        assert bad.nonzero().flatten().tolist() == [40, 130]
        m, v = (t.float() for t in moe.moe_adamw_moments(state))
        hit = torch.zeros(n, dtype=torch.bool, device="cuda")
        if bits == 32:
            hit[[40, 130]] = True
            assert torch.isnan(m[40]) and torch.isinf(m[130])
        else:  # the whole block of 32
            hit[32:64] = hit[128:160] = True
            assert torch.isnan(m[hit]).all() and torch.isnan(v[hit]).all()
            assert (state.exp_avg.scales == 255).nonzero().flatten().tolist() == [1, 4]
        assert torch.isfinite(m[~hit]).all() and torch.isfinite(v[~hit]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_large_ones(bits):
    """More tensors than a launch lists, one of them larger than all workgroups' first chunks: each as if stepped alone."""
    sizes = [1 + 37 * i % 700 for i in range(333)] + [20_000_003] + [64] * 3
    params, grads = tensors(sizes, (BF16, F32), 7), tensors(sizes, (F32, BF16), 8, 1e-2)
    alone = [p.clone() for p in params]
    state = moe.moe_adamw_state(params, bits=bits)
    moe.moe_adamw_step(state, grads, step=3, **HYPER)
    values = moe.moe_adamw_moments(state)
    for i in (0, 1, 79, 80, 81, 159, 160, 332, 333, 334, 336):
        one = moe.moe_adamw_state([alone[i]], bits=bits)
        moe.moe_adamw_step(one, [grads[i]], step=3, **HYPER)
        assert torch.equal(alone[i], params[i]), i
        for a, b in zip(values, moe.moe_adamw_moments(one)):
            assert torch.equal(a[place(state, i)], b[:sizes[i]]), i


def test_rate_step_and_scale_on_the_device():
    for bits, seed in ((32, None), (8, 3)):
        a, b = tensors([3000, 17], (BF16,), 9), tensors([3000, 17], (BF16,), 9)
        grads = tensors([3000, 17], (BF16,), 10)
        sa, sb = moe.moe_adamw_state(a, bits=bits), moe.moe_adamw_state(b, bits=bits)
        lr, step = torch.tensor([3e-3], device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda")
        scale = torch.tensor([0.25], device="cuda")
        rest = {k: v for k, v in HYPER.items() if k != "lr"}
        for t in (1, 2, 3):
            step += 1
            moe.moe_adamw_step(sa, grads, lr=float(lr.cpu()), step=t, seed=seed, **rest)
            moe.moe_adamw_step(sb, [g * 4 for g in grads], lr=lr, step=step, grad_scale=scale, seed=seed, **rest)
            assert all(torch.equal(x, y) for x, y in zip(a, b))
            assert all(torch.equal(x, y) for x, y in zip(moe.moe_adamw_moments(sa), moe.moe_adamw_moments(sb)))


def test_a_captured_step_counts_on():
    a, b = tensors([5000, 9], (BF16,), 11), tensors([5000, 9], (BF16,), 11)
    grads = tensors([5000, 9], (BF16,), 12)
    sa, sb = moe.moe_adamw_state(a, bits=8, master=True), moe.moe_adamw_state(b, bits=8, master=True)
    step = torch.tensor([0], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        moe.moe_adamw_step(sa, grads, step=step, seed=2, **HYPER)
    for t in range(1, 5):
        for g, fresh in zip(grads, tensors([5000, 9], (BF16,), 12 + t)):
            g.copy_(fresh)
        graph.replay()
        moe.moe_adamw_step(sb, grads, step=t, seed=2, **HYPER)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(sa.master, sb.master)
        assert torch.equal(sa.exp_avg.q, sb.exp_avg.q) and torch.equal(sa.exp_avg_sq.q, sb.exp_avg_sq.q)


def test_on_another_stream_and_as_parameters():
    p = torch.nn.Parameter(torch.ones((6, 40), device="cuda"))
    state = moe.moe_adamw_state([p])
    g = torch.ones((6, 40), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_adamw_step(state, [g], lr=0.1, weight_decay=0.0)
    torch.cuda.synchronize()
    assert torch.allclose(p, torch.full_like(p, 0.9), atol=1e-6, rtol=0)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_that_is_read_back(bits):
    """Moments, master and parameters may be other tensors from one step to the next, if they fit."""
    a, b = tensors([300, 64], (BF16,), 15), tensors([300, 64], (BF16,), 15)
    grads = tensors([300, 64], (BF16,), 16)
    sa, sb = (moe.moe_adamw_state(p, bits=bits, master=True) for p in (a, b))
    for t in (1, 2, 3):
        moe.moe_adamw_step(sa, grads, step=t, seed=1, **HYPER)
        moe.moe_adamw_step(sb, grads, step=t, seed=1, **HYPER)
        for p in b:
            p.data = p.data.clone()
        sb.master = sb.master.clone()
        for name in ("exp_avg", "exp_avg_sq"):
            m = getattr(sb, name)
            setattr(sb, name, m.clone() if bits == 32 else moe.Blocks8(m.q.clone(), m.scales.clone()))
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(sa.master, sb.master)
    m, short = sb.exp_avg, torch.zeros(96, device="cuda")
    for other in (short, moe.Blocks8(short.byte(), torch.zeros(3, dtype=torch.uint8, device="cuda")), None,
                  moe.moe_adamw_state(a, bits=40 - bits).exp_avg):
        sb.exp_avg = other
        for call in (lambda: moe.moe_adamw_step(sb, grads, step=4, **HYPER), lambda: moe.moe_adamw_moments(sb)):
            with pytest.raises((ValueError, TypeError)):
                call()
    sb.exp_avg, sb.master = m, short
    with pytest.raises(ValueError):
        moe.moe_adamw_step(sb, grads, step=4, **HYPER)
    sb.master = None
    flat = torch.zeros(400, dtype=BF16, device="cuda")
    b[0].data, b[1].data = flat[:300], flat[280:344]
    with pytest.raises(ValueError):
        moe.moe_adamw_step(sb, grads, step=4, **HYPER)


def test_refusals():
    p, g = tensors([64, 40], (BF16,), 13), tensors([64, 40], (BF16,), 14)
    state = moe.moe_adamw_state(p)
    for grads in (g[:1], [g[0], g[1][:39]], [g[0], g[1].cpu()], [g[0], torch.zeros(80, dtype=BF16, device="cuda")[::2]]):
        with pytest.raises(ValueError):
            moe.moe_adamw_step(state, grads, lr=1e-3)
    with pytest.raises(TypeError):
        moe.moe_adamw_step(state, [g[0], g[1].half()], lr=1e-3)
    for kw in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(weight_decay=-0.1), dict(lr=float("nan"))):
        with pytest.raises(moe.MoeError):
            moe.moe_adamw_step(state, g, **{"lr": 1e-3, **kw})
    for kw in (dict(seed=-1), dict(seed=1 << 32), dict(lr=torch.zeros(2, device="cuda")), dict(step=torch.ones(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            moe.moe_adamw_step(state, g, **{"lr": 1e-3, **kw})
    with pytest.raises(TypeError):
        moe.moe_adamw_step(state, g, lr=1e-3, step=torch.ones(1, device="cuda"))
    both = torch.zeros(96, dtype=BF16, device="cuda")
    for params in ([both, both], [both[:64], both[32:]], [both[::2]], [both, both.cpu()]):
        with pytest.raises(ValueError):
            moe.moe_adamw_state(params)
    m = torch.zeros(96, device="cuda")
    for args in ((m[:64], m), (m, moe.Blocks8(m, m)), (m, m, m[:32])):
        with pytest.raises((ValueError, TypeError)):
            moe.AdamW([both], *args)
    assert all(torch.equal(a, b) for a, b in zip(p, tensors([64, 40], (BF16,), 13)))  # nothing was stepped
