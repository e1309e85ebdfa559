"""MXFP4 products whose capacity, not the rows that are there, takes them to the pipelined tiles.

The host sees capacities alone: a buffer for many rows gets 256-row tiles however few of its rows have experts. So a
large capacity with small blocks reaches every way a tile can end: rows, columns and contraction inside a tile.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say
from test_gpu_mxfp4 import COUNTS, check_product, check_up

pytestmark = pytest.mark.gpu


def capacity(K, N, cols):
    """Rows from which a call of N output columns has too many small tiles of 32 rows and `cols` columns."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return 32 * (cus * (3 * (K + 256) + 3000) // ((K + 256) * -(-N // cols)) + 1)


@pytest.mark.parametrize("counts", COUNTS + [[0, 0], [300] * 20], ids=str)
@pytest.mark.parametrize("K,N", [(8, 8), (40, 72), (136, 264), (264, 40), (392, 520), (512, 256), (1032, 768)])
def test_projection(counts, K, N):
    say(f"[gpu] mxfp4 projection in a large buffer, rows={counts[:6]} K={K} N={N}")
    check_product(counts, K, N, spare=max(0, capacity(K, N, 64) - sum(counts)), seed=K + N)


@pytest.mark.parametrize("k,E,d,h", [(1, 1, 8, 8), (2, 3, 40, 24), (8, 128, 72, 40), (3, 7, 264, 136), (2, 4, 520, 264),
                                     (4, 9, 512, 128), (1, 2, 1032, 520), (2, 300, 96, 64)])
def test_up_swiglu(k, E, d, h):
    """Nearly every slot dropped: few sorted rows in a buffer for all of them."""
    kept = 1500 if E > 1 else 40
    T = -(-max(capacity(d, h, 32), 32 * E) // k)
    say(f"[gpu] mxfp4 gate/up in a large buffer, T={T} k={k} E={E} d={d} h={h}, {kept} kept")
    rng = np.random.default_rng(T + kept)
    ids = np.full(T * k, -1, np.int32)
    ids[rng.choice(T * k, kept, replace=False)] = rng.integers(0, E, kept)
    check_up(T, k, E, d, h, seed=d, ids=ids.reshape(T, k))


@pytest.mark.parametrize("d,h", [(72, 40), (264, 136), (520, 8), (512, 776)])
def test_up_swiglu_quantised(d, h):
    say(f"[gpu] mxfp4 gate/up to mxfp4 in a large buffer, d={d} h={h}")
    E, T = 6, capacity(d, h, 32)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(h)
    x = moe.moe_mxfp4_quantize(torch.randn((T, d), generator=g, device="cuda:0").bfloat16())
    w = moe.moe_mxfp4_quantize_weights(torch.randn((E, 2 * h, d), generator=g, device="cuda:0").bfloat16(), "out_in")
    x.scales[T // 3, 0] = 255  # a NaN row stays one
    counts = [257, 0, 1, 700, 31, 256]
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda:0")
    M = sum(counts)
    perm = torch.randperm(T, generator=g, device="cuda:0").int()
    perm[5] = T // 3
    want = moe.moe_mxfp4_quantize(moe.moe_gemm_up_swiglu_mxfp4(x, off, w, perm=perm)[:M].contiguous())
    q = torch.full((T, moe.mxfp4_row_bytes(h)), 0xAB, dtype=torch.uint8, device="cuda:0")
    s = torch.full((T, moe.mxfp4_scale_bytes(h)), 0xCD, dtype=torch.uint8, device="cuda:0")
    moe.moe_gemm_up_swiglu_mxfp4_q(x, off, w, perm=perm, q=q, scales=s)
    assert torch.equal(s[:M], want.scales) and torch.equal(q[:M], want.q) and (s[5, :-(-h // 32)] == 255).all()
    assert (q[M:] == 0xAB).all() and (s[M:] == 0xCD).all(), "rows past M were written"


@pytest.mark.parametrize("offsets", [[0, 1600, 1400, 9000], [700, 0, 1500, 1500], [-5, 10, 20, 2**31 - 1], [50000] * 4])
def test_offsets_outside_the_capacity(offsets):
    """Offsets are clamped into the capacity: nothing behind it is written, rows of one expert are its products."""
    K, N, E = 72, 40, 3
    cap = capacity(K, N, 64)
    say(f"[gpu] mxfp4 offsets {offsets} of {cap} rows")
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    x = moe.moe_mxfp4_quantize(torch.randn((cap, K), generator=g, device="cuda:0").bfloat16())
    w = moe.moe_mxfp4_quantize_weights(torch.randn((E, N, K), generator=g, device="cuda:0").bfloat16(), "out_in")
    buf = torch.full((cap + 64, N), 7.0, dtype=torch.bfloat16, device="cuda:0")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda:0")
    moe.moe_grouped_projection_mxfp4(x, off, w, y=buf[:cap])
    assert (buf[cap:] == 7.0).all()
    o = np.clip(offsets, 0, cap)
    hits = np.zeros(cap, np.int64)
    owner = np.zeros(cap, np.int64)
    for e in range(E):
        hits[o[e]:max(o[e], o[e + 1])] += 1
        owner[o[e]:max(o[e], o[e + 1])] = e
    none, one = torch.from_numpy(hits == 0).to("cuda:0"), torch.from_numpy(hits == 1).to("cuda:0")
    assert (buf[:cap][none] == 7.0).all()
    xv, wv = moe.moe_mxfp4_dequantize(x).double(), moe.moe_mxfp4_dequantize(w).double()
    W = wv[torch.from_numpy(owner).to("cuda:0")]
    want = (W * xv[:, None, :]).sum(2)
    tol = (W.abs() * xv.abs()[:, None, :]).sum(2) * (K / 2 + 64) * 2.0 ** -24
    err = (buf[:cap].double() - want).abs()
    assert (err <= tol + (want.abs() + tol) * 2.0 ** -8)[one].all()
