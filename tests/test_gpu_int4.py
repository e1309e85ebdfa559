"""4-bit experts with group scales on the GPU against 64 bits.

A result rounds once to bf16 (2^-8). The sums before it: a product s (A - (16 + z) B) is made of terms s (16 + q) x and
s (16 + z) x, each entering by at most K additions over the matrix instruction's lanes and steps, the groups and the four
waves, and a dozen roundings around them: (K + 16) 2^-24 of the sum of those magnitudes. SwiGLU's slopes are at most 1.1 and
the other factor; 16 more roundings of the result (exponential and reciprocal to an ulp or two).
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from oracle import int4 as oi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def u16(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def normal(shape, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(BF16)


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("E,K,N,group", [(1, 8, 8, 32), (2, 40, 24, 32), (3, 392, 520, 128), (2, 256, 64, 64), (1, 1000, 8, 128)])
def test_rounding_and_reading_back(layout, symmetric, E, K, N, group):
    w = normal((E, N, K), 1, 0.05)
    w[0, 1] = 0
    w[0, 2].abs_()
    w[0, 3, :5] = torch.tensor([-2.0, 1.0, 0.5, -0.25, 2.0])
    w[E - 1, 4, 7], w[E - 1, 5, 3], w[E - 1, 6, 1] = float("nan"), float("-inf"), 3e38
    given = w.transpose(1, 2).contiguous() if layout == "in_out" else w
    m = moe.moe_int4_quantize_weights(given, layout, group=group, symmetric=symmetric)
    back = moe.moe_int4_dequantize_weights(m)
    for e in range(E):
        q, s, z = oi.quantize(w[e].float().cpu().numpy(), group, symmetric)
        np.testing.assert_array_equal(m.q[e].cpu().numpy(), oi.pack(q))
        np.testing.assert_array_equal(u16(m.scales[e]), s)
        if symmetric:
            assert m.zeros is None
        else:
            np.testing.assert_array_equal(m.zeros[e].cpu().numpy(), z)
        v, _ = oi.values(q, s, z, group)
        want = torch.tensor(v).to(BF16)  # (12 bits: one rounding, of doubles that are exact)
        got = back[e].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def weights(E, N, K, group, zeros, seed=2):
    """Random codes, scales and zeros, the reference's values and magnitudes."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    G = -(-K // group)
    scales = torch.tensor(rng.uniform(0.01, 0.05, (E, G, N))).to(BF16).cuda()
    z = rng.integers(0, 16, (E, G, N)).astype(np.uint8) if zeros else None
    packed = np.stack([oi.pack(c) for c in codes])
    # what stands behind the last value is not used
    packed[..., -(-K // 2):] = rng.integers(0, 256, packed[..., -(-K // 2):].shape)
    m = moe.Int4(torch.tensor(packed).cuda(), scales, None if z is None else torch.tensor(z).cuda(), K, group)
    ref = [oi.values(codes[e], u16(scales[e]), None if z is None else z[e], group) for e in range(E)]
    return m, ref


def check(got, want, mag):
    err, tol = np.abs(f64(got) - want), 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * mag + 1e-38
    assert (err <= tol).all(), f"{(err / tol).max():.3g} times its tolerance"


def projection(counts, K, N, group, zeros, spare=0, seed=3):
    E, M = len(counts), sum(counts)
    m, ref = weights(E, N, K, group, zeros)
    x = normal((M + spare, K), seed)
    x[M:] = float("nan")  # rows behind the last are not read
    y = torch.full((M + spare, N), 7.0, dtype=BF16, device="cuda")
    off = offsets(counts)
    moe.moe_grouped_projection_int4(x, off, m, y=y)
    lo = 0
    for e, n in enumerate(counts):
        w, mag = ref[e]
        xe = f64(x[lo:lo + n])
        check(y[lo:lo + n], xe @ w.T, (K + 16) * U * (np.abs(xe) @ mag.T))
        lo += n
    assert (y[M:] == 7).all()


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [16, 17, 15, 1, 0, 33], [5, 0, 70, 31], [200]])
@pytest.mark.parametrize("K,N", [(8, 8), (40, 72), (128, 64), (392, 520), (776, 136)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_projection(counts, K, N, group, zeros):
    projection(counts, K, N, group, zeros, spare=2)


@pytest.mark.parametrize("K", [8, 16, 120, 136, 248, 504, 512, 520, 1032, 2880, 4104])
def test_contractions(K):
    projection([3, 0, 18], K, 40, 32, True)
    projection([40, 2], K, 40, 128, False)


def up(T, k, counts_of, E, d, h, group, zeros, drop=False, gather=True, seed=4):
    rng = np.random.default_rng(seed)
    m, ref = weights(E, 2 * h, d, group, zeros)
    x = normal((T, d), seed)
    S = T * k
    ids = rng.choice(E, S, p=counts_of)
    if drop:
        ids[rng.random(S) < 0.3] = E
    order = np.argsort(ids, kind="stable")
    counts = np.bincount(ids, minlength=E + 1)[:E]
    M = counts.sum()
    perm = torch.tensor(order, dtype=torch.int32, device="cuda")
    out = torch.full((S, h), 7.0, dtype=BF16, device="cuda")
    if gather:
        moe.moe_gemm_up_swiglu_int4(x, offsets(counts), m, perm=perm, k=k, h_buf=out)
        rows = f64(x)[order // k]
    else:
        xs = x[(perm // k).long()].contiguous()
        moe.moe_gemm_up_swiglu_int4(xs, offsets(counts), m, h_buf=out)
        rows = f64(xs)
    lo = 0
    for e in range(E):
        n = counts[e]
        w, mag = ref[e]
        xe = rows[lo:lo + n]
        u, du = xe @ w.T, (d + 16) * U * (np.abs(xe) @ mag.T)
        g, dg, u, du = u[:, :h], du[:, :h], u[:, h:], du[:, h:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        check(out[lo:lo + n], silu * u, 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 16 * U * np.abs(silu * u))
        lo += n
    assert (out[M:] == 7).all()


@pytest.mark.parametrize("T,k,E,d,h,group,zeros", [
    (1, 1, 1, 64, 32, 32, False), (4, 8, 128, 256, 40, 64, False), (4, 2, 8, 392, 104, 128, True), (9, 3, 4, 136, 8, 32, True),
    (100, 2, 5, 160, 72, 64, True), (300, 1, 3, 96, 56, 128, False)])
@pytest.mark.parametrize("gather", [True, False])
def test_gate_up(T, k, E, d, h, group, zeros, gather):
    p = np.arange(1, E + 1) ** -1.0
    up(T, k, p / p.sum(), E, d, h, group, zeros, gather=gather)
    up(T, k, p / p.sum(), E, d, h, group, zeros, drop=True, gather=gather)


@pytest.mark.parametrize("rows", [1000, 4000, 10000])  # tiles of 32 and, twice, of 64 rows
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("K", [264, 512])
def test_wide_tiles(rows, group, zeros, K):
    projection([0, 1, 65, rows - 131, 33, 32], K, 2056, group, zeros, spare=1)
    p = np.array([0.001, 0.9, 0.02, 0.06, 0.019])
    up(rows // 2, 2, p, 5, K, 1032, group, zeros, drop=group == 64)


def test_many_experts():
    rng = np.random.default_rng(5)
    for E in (255, 256, 257, 1024):
        projection(rng.integers(0, 3, E).tolist(), 32, 8, 32, False)


@pytest.mark.parametrize("rows", [40000, 70000])  # tiles of 32 and of 64 rows, tables of as many experts as there can be
def test_wide_tiles_of_many_experts(rows):
    rng = np.random.default_rng(rows)
    p = np.arange(1, 1025) ** -0.5
    projection(rng.multinomial(rows, p / p.sum()).tolist(), 64, 64, 32, True, spare=5)


@pytest.mark.parametrize("rows", [40, 1000, 10000])  # each kind of tile
def test_what_is_not_finite_stays_in_its_row_and_column(rows):
    m, _ = weights(2, 2056, 264, 64, True)
    x, off = normal((rows, 264), 20), offsets([rows // 2, rows - rows // 2])
    clean = moe.moe_grouped_projection_int4(x, off, m)
    x[3, 7], x[rows - 2, 263] = float("nan"), float("inf")
    m.scales[1, 4, 2050] = float("nan")
    got = moe.moe_grouped_projection_int4(x, off, m)
    assert torch.isnan(got[[3, rows - 2]]).all() and torch.isnan(got[rows // 2:, 2050]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[[3, rows - 2]] = False
    keep[rows // 2:, 2050] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("rows", [1000, 10000])
def test_bad_offsets_stay_inside_wide_tiles(rows):
    m, ref = weights(3, 2056, 264, 32, True)
    x, y = normal((rows, 264), 21), torch.full((rows, 2056), 7.0, dtype=BF16, device="cuda")
    off = torch.tensor([-9, rows - 100, rows // 2, 1 << 30], dtype=torch.int32, device="cuda")
    moe.moe_grouped_projection_int4(x, off, m, y=y)
    want = moe.moe_grouped_projection_int4(x, torch.tensor([0, rows // 2, rows // 2, rows], dtype=torch.int32, device="cuda"), m)
    # rows from rows / 2 to rows - 100 belong to two experts
    assert torch.equal(y[:rows // 2], want[:rows // 2]) and torch.equal(y[rows - 100:], want[rows - 100:])


def test_bad_offsets_stay_inside():
    """Offsets past the capacity are cut, an expert whose end precedes its start is empty, and nothing else is written."""
    m, ref = weights(3, 16, 32, 32, True)
    x, y = normal((6, 32), 6), torch.full((6, 16), 7.0, dtype=BF16, device="cuda")
    off = torch.tensor([0, 4, 2, 99], dtype=torch.int32, device="cuda")
    moe.moe_grouped_projection_int4(x, off, m, y=y)
    xe = f64(x)
    w0, g0 = ref[0]
    w2, g2 = ref[2]
    first = 48 * U
    check(y[:2], xe[:2] @ w0.T, first * (np.abs(xe[:2]) @ g0.T))
    check(y[4:], xe[4:] @ w2.T, first * (np.abs(xe[4:]) @ g2.T))
    y.fill_(7.0)
    moe.moe_grouped_projection_int4(x, torch.tensor([-5, -1, -1, -1], dtype=torch.int32, device="cuda"), m, y=y)
    assert (y == 7).all()


def test_no_rows_and_unused_capacity():
    m, _ = weights(2, 16, 32, 32, False)
    e = torch.empty((0, 32), dtype=BF16, device="cuda")
    assert moe.moe_grouped_projection_int4(e, offsets([0, 0]), m).shape == (0, 16)
    y = torch.full((500, 16), 7.0, dtype=BF16, device="cuda")
    x = normal((500, 32), 7)
    moe.moe_grouped_projection_int4(x, offsets([0, 0]), m, y=y)
    assert (y == 7).all()
    # the capacity chooses the tiles, the rows decide the result: close whatever the spare rows
    few = moe.moe_grouped_projection_int4(x[:3].contiguous(), offsets([1, 2]), m)
    moe.moe_grouped_projection_int4(x, offsets([1, 2]), m, y=y)
    assert torch.equal(y[:3], few)


def test_whole_step_streams_and_a_graph():
    T, k, E, d, h = 6, 2, 8, 128, 64
    w_ug, w_down = normal((E, 2 * h, d), 8, 0.1), normal((E, h, d), 9, 0.1)
    u4 = moe.moe_int4_quantize_weights(w_ug, "out_in", group=64)
    d4 = moe.moe_int4_quantize_weights(w_down, "in_out", group=32, symmetric=True)
    x, logits = normal((T, d), 10), normal((T, E), 11)
    r = moe.moe_router_topk(logits, k)

    def parts():
        p = moe.moe_permute(x, r.expert_ids, E)
        hb = moe.moe_gemm_up_swiglu_int4(p.x_perm, p.offsets, u4)
        return moe.moe_unpermute(moe.moe_grouped_projection_int4(hb, p.offsets, d4), p.inv_map, r.routing_w)

    y, _ = moe.moe_expert_forward_int4(x, r.expert_ids, r.routing_w, u4, d4)
    assert torch.equal(y, parts())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, _ = moe.moe_expert_forward_int4(x, r.expert_ids, r.routing_w, u4, d4)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = moe.moe_expert_forward_int4(x, r.expert_ids, r.routing_w, u4, d4)
    for seed in (10, 12, 13):
        x.copy_(normal((T, d), seed))
        graph.replay()
        want = parts()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    m, _ = weights(2, 16, 64, 32, True)
    x, off = normal((4, 64), 14), offsets([2, 2])
    S = moe.Int4
    for bad in (S(m.q, m.scales, m.zeros, 64, 16), S(m.q, m.scales, m.zeros, 64, 64), S(m.q, m.scales, m.zeros, 96, 32),
                S(m.q[:, :8], m.scales, m.zeros, 64, 32), S(m.q, m.scales, m.zeros.cpu(), 64, 32),
                S(m.q[0], m.scales, m.zeros, 64, 32)):
        with pytest.raises(ValueError):
            moe.moe_grouped_projection_int4(x, off, bad)
    for call in (lambda: moe.moe_grouped_projection_int4(x[:, :32].contiguous(), off, m),
                 lambda: moe.moe_grouped_projection_int4(x, off[:2], m), lambda: moe.moe_grouped_projection_int4(x[0], off, m),
                 lambda: moe.moe_gemm_up_swiglu_int4(x, off, m, k=2),
                 lambda: moe.moe_gemm_up_swiglu_int4(x, off, m, perm=off, k=2),
                 lambda: moe.moe_int4_quantize_weights(normal((1, 8, 64), 1), "out_in", group=16),
                 lambda: moe.moe_int4_quantize_weights(normal((1, 8, 64), 1), "out_in", symmetric=True, zeros=m.zeros)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_grouped_projection_int4(x.float(), off, m), lambda: moe.moe_grouped_projection_int4(x, off, x),
                 lambda: moe.moe_grouped_projection_int4(x, off, S(m.q, m.scales.float(), m.zeros, 64, 32))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(moe.MoeError):  # rows of no multiple of 8 values
        moe.moe_grouped_projection_int4(x[:, :60].contiguous(), off, S(m.q, m.scales, m.zeros, 60, 32))
