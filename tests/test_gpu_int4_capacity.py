"""4-bit products whose buffers hold far more rows than there are: the capacity chooses the kind of tile, few rows run on
wide ones. Tolerances as for full buffers; rows behind the last sequence stay as they were.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from test_gpu_int4 import BF16, U, check, f64, normal, offsets, weights

pytestmark = pytest.mark.gpu

# capacities whose estimated times (3 units, tiles of 256 weight rows) choose tiles of 16, 32 and 64 rows
CAPACITIES = [40, 1000, 10000]


def up_columns(x, ref, h, K):
    """SiLU(g) u in 64 bits and what fp32 sums may be off by, rows x of one expert."""
    w, mag = ref
    v, dv = x @ w.T, (K + 16) * U * (np.abs(x) @ mag.T)
    g, dg, u, du = v[:, :h], dv[:, :h], v[:, h:], dv[:, h:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    return silu * u, 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 16 * U * np.abs(silu * u)


@pytest.mark.parametrize("capacity", CAPACITIES)
@pytest.mark.parametrize("counts", [[1, 2], [0, 3], [0, 0], [17, 16]])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_few_rows_in_a_large_buffer(capacity, counts, group, zeros):
    K, N, M = 264, 2056, sum(counts)
    m, ref = weights(2, N, K, group, zeros)
    x = normal((capacity, K), 31)
    x[M:] = float("nan")  # rows behind the last are not read
    y = torch.full((capacity, N), 7.0, dtype=BF16, device="cuda")
    moe.moe_grouped_projection_int4(x, offsets(counts), m, y=y)
    lo = 0
    for e, n in enumerate(counts):
        xe = f64(x[lo:lo + n])
        check(y[lo:lo + n], xe @ ref[e][0].T, (K + 16) * U * (np.abs(xe) @ ref[e][1].T))
        lo += n
    assert (y[M:] == 7).all()


@pytest.mark.parametrize("capacity", CAPACITIES)
@pytest.mark.parametrize("counts", [[1, 2], [0, 3], [17, 16]])
@pytest.mark.parametrize("gather", [True, False])
def test_few_rows_of_gate_and_up_in_a_large_buffer(capacity, counts, gather):
    K, h, group, k, M = 264, 1032, 64, 2, sum(counts)
    m, ref = weights(2, 2 * h, K, group, True)
    out = torch.full((capacity, h), 7.0, dtype=BF16, device="cuda")
    if gather:
        x = normal((capacity // k, K), 32)
        perm = torch.arange(capacity - 1, -1, -1, dtype=torch.int32, device="cuda")
        moe.moe_gemm_up_swiglu_int4(x, offsets(counts), m, perm=perm, k=k, h_buf=out)
        rows = f64(x[(perm[:M] // k).long()])
    else:
        x = normal((capacity, K), 32)
        x[M:] = float("nan")
        moe.moe_gemm_up_swiglu_int4(x, offsets(counts), m, h_buf=out)
        rows = f64(x[:M])
    lo = 0
    for e, n in enumerate(counts):
        check(out[lo:lo + n], *up_columns(rows[lo:lo + n], ref[e], h, K))
        lo += n
    assert (out[M:] == 7).all()


# widths that leave a wide tile's last waves without a column of their own
@pytest.mark.parametrize("N", [72, 264, 520])
@pytest.mark.parametrize("rows", [9000, 40000])
def test_widths_that_end_inside_a_wide_tile(N, rows):
    K, counts = 136, [rows // 3, 1, rows - rows // 3 - 1]
    m, ref = weights(3, N, K, 32, True)
    x = normal((rows, K), 33)
    y = moe.moe_grouped_projection_int4(x, offsets(counts), m)
    lo = 0
    for e, n in enumerate(counts):
        xe = f64(x[lo:lo + n])
        check(y[lo:lo + n], xe @ ref[e][0].T, (K + 16) * U * (np.abs(xe) @ ref[e][1].T))
        lo += n
    if N % 16:
        return
    h = N // 2
    out = moe.moe_gemm_up_swiglu_int4(x, offsets(counts), m)
    lo = 0
    for e, n in enumerate(counts):
        check(out[lo:lo + n], *up_columns(f64(x[lo:lo + n]), ref[e], h, K))
        lo += n
