"""MXFP4 scale bytes at both ends of their range, as another quantiser may write them (on an MI355X).

A bf16 number holds a 4-bit value times 2^e exactly while it is finite: down to 0.5 * 2^-127, a subnormal, and up to scale
byte 252 for every value. Above that the value reads back as the bf16 it rounds to, which past the largest finite one is
an infinity. Products: tolerances as in test_gpu_mxfp4.py, every product being a normal fp32 number here.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import say, to_dev
from oracle import mxfp4 as om
from test_gpu_mxfp4 import sums
from test_gpu_mxfp4_capacity import capacity

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CODES = np.arange(16, dtype=np.uint8)
TOP = 2.0 ** 128 - 2.0 ** 119  # halfway from the largest finite bf16 to 2^128: from here a value rounds to infinity


def every_code(byte):
    """A row of one block that holds every code twice."""
    row = np.concatenate([CODES, CODES])
    return row[0::2] | (row[1::2] << 4), byte


def test_reading_back_every_code_at_every_scale():
    say("[gpu] mxfp4 read back: every code at every scale byte")
    q = np.stack([every_code(b)[0] for b in range(256)])
    s = np.zeros((256, 16), np.uint8)
    s[:, 0] = np.arange(256)
    got = moe.moe_mxfp4_dequantize(moe.Mxfp4(to_dev(q), to_dev(s), 32)).double().cpu().numpy()
    want = om.dequantize(q, s, 32)
    assert np.isnan(got[255]).all()
    over = np.abs(want[:255]) >= TOP
    assert not over[:253].any() and over[253].sum() == 8 and over[254].sum() == 16  # 4, 6 and 2, 3, 4, 6, both signs, twice
    want[:255] = np.where(over, np.copysign(np.inf, want[:255]), want[:255])
    np.testing.assert_array_equal(got[:255], want[:255])


def codes_with_scales(rng, shape, K, lo, hi):
    q = rng.integers(0, 256, size=(*shape, om.row_bytes(K)), dtype=np.uint8)
    s = rng.integers(lo, hi + 1, size=(*shape, om.scale_bytes(K)), dtype=np.uint8)
    cut = np.arange(om.row_bytes(K) * 2) < K  # zeros behind the last value
    q &= (cut[0::2] * 15 + cut[1::2] * 240).astype(np.uint8)
    return moe.Mxfp4(to_dev(q), to_dev(s), K), om.dequantize(q, s, K)


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("x_bytes,w_bytes", [((0, 2), (252, 254)), ((252, 254), (0, 2)), ((20, 40), (214, 234))])
@pytest.mark.parametrize("K,N", [(64, 72), (136, 40), (512, 128)])
def test_products_of_far_scales(K, N, x_bytes, w_bytes, large):
    say(f"[gpu] mxfp4 products of scale bytes {x_bytes} and {w_bytes}, K={K} N={N}, large={large}")
    rng = np.random.default_rng(K + x_bytes[0])
    counts = [5, 0, 300, 33]
    E, M = len(counts), sum(counts)
    rows = max(M, capacity(K, N, 64)) if large else M
    x, xv = codes_with_scales(rng, (rows,), K, *x_bytes)
    w, wv = codes_with_scales(rng, (E, N), K, *w_bytes)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = moe.moe_grouped_projection_mxfp4(x, to_dev(off), w).double().cpu().numpy()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        want, tol = sums(xv[lo:hi], wv[e])
        assert (np.abs(y[lo:hi] - want) <= tol + (np.abs(want) + tol) * 2.0 ** -8).all(), e
