"""Pins of the 64-bit norms, AdamW with its 8-bit moments, and 4-bit weights: autograd, formats, rounding (no GPU)."""

import numpy as np
import pytest
import torch

from oracle import adamw as oa
from oracle import int4 as oi
from oracle import norm as on


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("nxt", [False, True])
def test_norm_backward_is_autograd_of_the_forward(post, gate, nxt):
    rng = np.random.default_rng(3)
    T, d, a, b, eps = 5, 12, 0.9, 0.4, 1e-3
    r, y = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    wp, wn = 1 + 0.3 * rng.normal(size=d), 1 + 0.3 * rng.normal(size=d)
    gv = {"none": np.ones(1), "token": rng.random((T, 1)), "channel": rng.normal(size=d)}[gate]
    kw = dict(post=post, w_post=wp, gate=gv, a=a, b=b, nxt=nxt, w_next=wn, eps=eps)
    x, n, _, _ = on.forward(r, y, **kw)
    dr, dn = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    got = on.backward(dr, dn, x, y, gate_kind=gate, **kw)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(r=r, y=y, w_post=wp, w_next=wn, gate=gv).items()}

    def unit(v):
        return v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + eps)

    u = unit(t["y"]) * t["w_post"] if post else t["y"]
    tx = a * t["r"] + b * t["gate"] * u
    np.testing.assert_allclose(tx.detach().numpy(), x, rtol=1e-13, atol=1e-14)
    total = (tx * torch.tensor(dr)).sum()
    if nxt:
        tn = unit(tx) * t["w_next"]
        np.testing.assert_allclose(tn.detach().numpy(), n, rtol=1e-13, atol=1e-14)
        total = total + (tn * torch.tensor(dn)).sum()
    total.backward()
    assert set(got) == {"r", "y"} | ({"w_next"} if nxt else set()) | ({"w_post"} if post else set()) | (
        {"gate"} if gate != "none" else set())
    for k, (v, mag) in got.items():
        np.testing.assert_allclose(v, t[k].grad.numpy(), rtol=1e-11, atol=1e-13)
        assert (mag >= np.abs(v) * (1 - 1e-12)).all()


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(4)
    x, w, dn = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=(3, 8))
    got = on.backward(None, dn, x, w_next=w)["r"][0]
    for t, c in ((0, 0), (1, 5), (2, 7)):
        step = np.zeros_like(x)
        step[t, c] = 1e-5
        up, down = on.forward(x + step, w_next=w)[1], on.forward(x - step, w_next=w)[1]
        assert abs(((up - down) * dn).sum() / 2e-5 - got[t, c]) < 1e-8


def test_step_is_torch_adamw():
    rng = np.random.default_rng(5)
    p, m, v = rng.normal(size=50), rng.normal(size=50) * 1e-2, rng.random(50) * 1e-4
    t = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.99), eps=1e-6, weight_decay=0.3)
    opt.state[t] = dict(step=torch.tensor(6.0), exp_avg=torch.tensor(m), exp_avg_sq=torch.tensor(v))
    g = rng.normal(size=50)
    t.grad = torch.tensor(g)
    opt.step()
    q, m2, v2, _ = oa.step64(p, g, m, v, lr=1e-2, b1=0.8, b2=0.99, eps=1e-6, wd=0.3, t=7)
    np.testing.assert_allclose(q, t.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(m2, opt.state[t]["exp_avg"].numpy(), rtol=1e-12)
    np.testing.assert_allclose(v2, opt.state[t]["exp_avg_sq"].numpy(), rtol=1e-12)


def test_e4m3_is_torch_float8():
    values = oa.e4m3_values()
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(values, codes)
    rng = np.random.default_rng(6)
    m = (rng.normal(size=(200, 32)) * np.exp2(rng.integers(-20, 1, size=(200, 32)))).astype(np.float32)
    q, s = oa.to_e4m3(m.reshape(-1))
    scaled = torch.tensor(m.astype(np.float64) * np.exp2(127.0 - s.astype(float))[:, None])
    assert 128 <= scaled.abs().max() < 256
    want = scaled.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(-1)
    np.testing.assert_array_equal(q, want)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 90])
def test_codes_read_back_as_themselves(scale):
    e5, e4 = oa.e5m3_values(), oa.e4m3_values()
    assert (np.diff(e5) > 0).all() and (np.diff(e4) > 0).all()
    v = np.append(e5[:248], np.zeros(8)).reshape(-1, 32)
    v[:, 0] = e5[247]  # every block reaches the top
    v = (v * scale).astype(np.float32).reshape(-1)
    q, s = oa.to_e5m3(v)
    np.testing.assert_array_equal(oa.of_e5m3(q, s).astype(np.float32), v)
    m = np.append(e4[:120], -e4[:104]).reshape(-1, 32)
    m[:, 0] = e4[119]
    m = (m * scale).astype(np.float32).reshape(-1)
    q, s = oa.to_e4m3(m)
    np.testing.assert_array_equal(oa.of_e4m3(q, s).astype(np.float32), m)


def test_second_moments_keep_what_is_above_zero():
    v = np.zeros(64, np.float32)
    v[0], v[1], v[2] = 1.0, 1e-30, 1e-42
    v[32:] = np.nan
    q, s = oa.to_e5m3(v)
    assert q[0] == 240 and q[1] == 1 and q[2] == 1 and not q[3:].any() and s[1] == 255
    assert np.isnan(oa.of_e5m3(q, s)[32:]).all()


def test_random_rounding_has_the_right_mean():
    """Of 2^16 places, an up-rounding of probability f happens 2^16 f times within five standard deviations."""
    bits = oa.random_bits(7, 3, np.arange(1 << 16))
    for part in (bits & 0xFFFF, bits >> 16):
        for f in (0.01, 0.25, 0.5, 0.9):
            got = ((part + int(f * 65536)) >= 65536).mean()
            assert abs(got - f) < 5 * np.sqrt(f * (1 - f) / 65536) + 2 ** -16
    other = oa.random_bits(7, 4, np.arange(1 << 16))
    for a, b in (((bits & 0xFFFF), bits >> 16), (bits & 0xFFFF, other & 0xFFFF), (bits[:-1] >> 16, bits[1:] >> 16)):
        assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 256


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("group", [32, 128])
def test_int4_values_are_within_half_a_step(symmetric, group):
    rng = np.random.default_rng(8)
    w = rng.normal(size=(24, 200)).astype(np.float32)
    w[3] = 0
    w[4, :40] = np.abs(w[4, :40])
    q, s, z = oi.quantize(w, group, symmetric)
    np.testing.assert_array_equal(oi.unpack(oi.pack(q), 200), q)
    v, _ = oi.values(q, s, z, group)
    step = oi.values(np.ones_like(q), s, np.zeros_like(s, dtype=np.uint8), group)[0]
    # half a step, and what the codes at the ends lose to the scale's own rounding (bf16, 2^-8 of the range) and to z's
    slack = step * (7 if symmetric else 15) * 2.0 ** -8 + (0 if symmetric else step / 2)
    assert (np.abs(v - w) <= step / 2 + slack + 1e-12).all()
    assert (v[3] == 0).all()
