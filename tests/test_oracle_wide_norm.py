"""The reference's norm gradient for wide rows against the one through the Jacobian."""

import numpy as np
import pytest

from oracle import norm as on


@pytest.mark.parametrize("T,d", [(1, 8), (3, 40), (5, 264)])
@pytest.mark.parametrize("post,gate,nxt", [(True, "channel", True), (False, "token", True), (True, "none", False)])
def test_closed_form_is_the_jacobian_s_product(T, d, post, gate, nxt):
    rng = np.random.default_rng(T * d)
    x, y, dr, dn = (rng.standard_normal((T, d)) for _ in range(4))
    kw = dict(post=post, w_post=rng.uniform(0.5, 1.5, d), w_next=rng.uniform(0.5, 1.5, d), a=0.75, b=1.5, nxt=nxt, eps=1e-5,
              gate={"none": 1.0, "token": rng.standard_normal((T, 1)), "channel": rng.standard_normal(d)}[gate], gate_kind=gate)
    want = on.backward(dr, dn, x, y, **kw)
    got = on.backward(dr, dn, x, y, through=on.through_wide_norm, **kw)
    assert set(got) == set(want)
    for k in want:  # doubles: sums of d (and T) terms
        for a, b in zip(got[k], want[k]):
            assert (np.abs(a - b) <= (4 * d + T + 50) * 2.0 ** -53 * (want[k][1] + np.abs(want[k][1]).max())).all(), k
