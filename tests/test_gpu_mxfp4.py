"""MXFP4 kernels against the 64-bit reference, on an MI355X.

Quantising and reading back are exact: codes, scale bytes and values are compared bit for bit (the sign of a zero
aside: -0 and 0 are one value). A product of two MXFP4 rows is a sum of K exact terms in fp32: it is off by at most
(K / 2 + 64) 2^-24 of the terms' magnitudes (pairs are summed exactly or rounded once, then added one by one), plus
half a bf16 step, 2^-8 of the result. SwiGLU h = SiLU(g) u of such sums carries their errors with slopes at most
1.1 |u| and |SiLU(g)|, and (|g| + 16) 2^-22 of its own from the exponential and reciprocal.
"""

import numpy as np
import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe
from gpu_util import bits, say, to_dev
from oracle import mxfp4 as om
from oracle.bf16 import bf16_bits_to_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def codes_of(q):
    """Codes with the sign of a zero dropped."""
    q = np.asarray(q)
    c = np.stack([q & 15, q >> 4], axis=-1)
    return np.where(c == 8, 0, c)


def check_quantize(x, m, rows_first=None):
    q, s = om.quantize(x)
    np.testing.assert_array_equal(m.scales.cpu().numpy().reshape(s.shape), s)
    np.testing.assert_array_equal(codes_of(m.q.cpu().numpy().reshape(q.shape)), codes_of(q))
    v = moe.moe_mxfp4_dequantize(m).double().cpu().numpy().reshape(x.shape)
    np.testing.assert_array_equal(v, om.dequantize(q, s, x.shape[1]))


def test_quantize_every_bf16_value():
    """Every bf16 pattern as its block's largest, beside smaller ones; then every pattern below a few largest."""
    say("[gpu] mxfp4 quantise: every bf16 value")
    rng = np.random.default_rng(0)
    pat = np.arange(65536, dtype=np.uint16)
    x = np.repeat(pat[:, None], 32, axis=1)
    # the other values: the same pattern with up to 5 exponents less and any mantissa, either sign
    ex, mant = (pat >> 7) & 255, rng.integers(0, 128, size=x.shape)
    drop = rng.integers(1, 6, size=x.shape)
    other = (np.maximum(ex[:, None].astype(np.int64) - drop, 0) << 7 | mant | rng.integers(0, 2, size=x.shape) << 15)
    at = np.arange(32)[None, :] == (pat[:, None] % 32)
    x = np.where(at, x, other).astype(np.uint16)
    t = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
    check_quantize(bf16_bits_to_f64(x), moe.moe_mxfp4_quantize(t.to(DEV)))
    for top in (0x0001, 0x007F, 0x0080, 0x0100, 0x0180, 0x01FF, 0x3F80, 0x40FF, 0x7F00, 0x7F7F):
        mags = np.arange(top + 1, dtype=np.uint16)
        mags = np.concatenate([mags, mags | 0x8000])
        mags = np.concatenate([mags, np.zeros(-len(mags) % 31, np.uint16)]).reshape(-1, 31)
        x = np.concatenate([np.full((len(mags), 1), top, np.uint16), mags], axis=1)
        t = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
        check_quantize(bf16_bits_to_f64(x), moe.moe_mxfp4_quantize(t.to(DEV)))


@pytest.mark.parametrize("R,K", [(1, 8), (3, 24), (5, 32), (7, 40), (2, 504), (33, 512), (9, 520), (1, 2880), (1000, 136),
                                 (257, 2048), (3, 70000), (5000, 8)])
def test_quantize_rows(R, K):
    say(f"[gpu] mxfp4 quantise rows={R} K={K}")
    rng = np.random.default_rng(R + K)
    x = bf16(rng.normal(size=(R, K)) * np.exp(rng.normal(size=(R, K)) * 2))
    x[0, 0] = 0.0
    x[R // 2, K // 2] = float("inf")
    x[-1, -1] = float("nan")
    m = moe.moe_mxfp4_quantize(x.to(DEV), q=torch.full((R, moe.mxfp4_row_bytes(K)), 0xAB, dtype=torch.uint8, device=DEV),
                               scales=torch.full((R, moe.mxfp4_scale_bytes(K)), 0xFF, dtype=torch.uint8, device=DEV))
    check_quantize(x.double().numpy(), m)


@pytest.mark.parametrize("E,d_in,d_out", [(1, 8, 8), (3, 24, 40), (2, 136, 264), (1, 2880, 72), (5, 520, 128), (2, 40, 1000)])
def test_quantize_weights_both_layouts(E, d_in, d_out):
    say(f"[gpu] mxfp4 weights E={E} {d_in} -> {d_out}")
    rng = np.random.default_rng(E + d_in)
    w = bf16(rng.normal(size=(E, d_in, d_out)) * 0.05)
    w[0, 0, 1] = float("nan")
    wd = w.to(DEV)
    a = moe.moe_mxfp4_quantize_weights(wd, "in_out")
    b = moe.moe_mxfp4_quantize_weights(wd.transpose(1, 2).contiguous(), "out_in")
    assert torch.equal(a.q, b.q) and torch.equal(a.scales, b.scales) and a.width == d_in
    check_quantize(w.transpose(1, 2).reshape(E * d_out, d_in).double().numpy(), a)


def test_quantize_nothing():
    m = moe.moe_mxfp4_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert m.q.shape == (0, 32) and moe.moe_mxfp4_dequantize(m).shape == (0, 64)


# ------------------------------------------------------------------ products


def packed(rng, shape, sigma=1.0):
    """(Mxfp4 on the device, its float64 values): random codes with scales of several sizes, as quantised rows have."""
    K = shape[-1]
    R = int(np.prod(shape[:-1]))
    x = rng.normal(size=(R, K)) * sigma * np.exp2(rng.integers(-2, 3, size=(R, 1)))
    q, s = om.quantize(x)
    v = om.dequantize(q, s, K)
    # what stands behind the last value and the last block must not matter
    s[:, -(-K // 32):] = 0xFF
    m = moe.Mxfp4(to_dev(q.reshape(*shape[:-1], -1)), to_dev(s.reshape(*shape[:-1], -1)), K)
    return m, v.reshape(shape)


def sums(x, w):
    """(x w^T, the bound on its fp32 error)."""
    K = x.shape[1]
    return x @ w.T, (np.abs(x) @ np.abs(w).T) * (K / 2 + 64) * U


def silu(g):
    return g / (1.0 + np.exp(-g))


def check_product(counts, K, N, spare=0, seed=0):
    rng = np.random.default_rng(seed)
    E, M = len(counts), int(sum(counts))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xv = packed(rng, (M + spare, K))
    w, wv = packed(rng, (E, N, K), 0.1)
    y = torch.full((M + spare, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_projection_mxfp4(x, to_dev(offsets), w, y=y)
    got = y.double().cpu().numpy()
    assert (got[M:] == 7.0).all(), "rows past M were written"
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        want, tol = sums(xv[lo:hi], wv[e])
        err = np.abs(got[lo:hi] - want)
        bad = err > tol + (np.abs(want) + tol) * 2.0 ** -8
        assert not bad.any(), (e, np.argwhere(bad)[:5], err[bad][:5], want[bad][:5])


def check_up(T, k, E, d, h, seed=0, drop=0.1, ids=None):
    rng = np.random.default_rng(seed)
    if ids is None:
        ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
        ids[rng.random((T, k)) < drop] = -1
    x, xv = packed(rng, (T, d))
    w, wv = packed(rng, (E, 2 * h, d), 0.1)
    p = moe.moe_permute(torch.zeros((T, 8), dtype=torch.bfloat16, device=DEV), to_dev(ids), E, gather=False)
    out = torch.full((T * k, h), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_up_swiglu_mxfp4(x, p.offsets, w, perm=p.perm, k=k, h_buf=out)
    offsets, perm = p.offsets.cpu().numpy(), p.perm.cpu().numpy()
    got = out.double().cpu().numpy()
    M = offsets[-1]
    assert (got[M:] == 7.0).all(), "rows past M were written"
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        s, tol = sums(xv[perm[lo:hi] // k], wv[e])
        g, u, tg, tu = s[:, :h], s[:, h:], tol[:, :h], tol[:, h:]
        want = silu(g) * u
        t = 1.1 * (np.abs(u) + tu) * tg + np.abs(silu(g)) * tu + np.abs(want) * (np.abs(g) + 16) * 2.0 ** -22
        err = np.abs(got[lo:hi] - want)
        assert (err <= t + (np.abs(want) + t) * 2.0 ** -8 + 2.0 ** -126).all(), (e, (err - t).max())
    # the same rows already in sorted order, without perm
    rows = torch.from_numpy((perm[:M] // k).astype(np.int64)).to(DEV)
    sorted_x = moe.Mxfp4(x.q[rows].contiguous(), x.scales[rows].contiguous(), d)
    plain = torch.full((M, h), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_up_swiglu_mxfp4(sorted_x, p.offsets, w, h_buf=plain)
    np.testing.assert_array_equal(bits(plain), bits(out)[:M])


COUNTS = [[1], [0, 1, 0], [32, 0, 33, 31, 1], [5, 64, 0, 200], [129, 255, 1, 257, 0, 63]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(8, 8), (32, 24), (40, 72), (64, 64), (136, 264), (256, 256), (264, 40), (392, 520), (768, 128)])
def test_projection(counts, K, N):
    say(f"[gpu] mxfp4 projection rows={counts} K={K} N={N}")
    check_product(counts, K, N, spare=3, seed=K + N)


@pytest.mark.parametrize("counts,K,N", [
    ([400, 0, 700, 513], 512, 256), ([1000, 1], 520, 512), ([2100], 2880, 264), ([3, 900, 64, 1500], 1032, 768),
    ([700] * 8, 256, 512), ([511, 512, 513, 769] * 3, 768, 1024), ([450] * 40, 64, 64), ([256] * 16, 2048, 256),
    ([150] * 16, 2056, 264), ([40] * 64, 768, 512), ([17] * 100, 520, 136), ([2] * 1024, 96, 32),
])
def test_projection_many_rows(counts, K, N):
    say(f"[gpu] mxfp4 projection rows={counts[:4]}... K={K} N={N}")
    check_product(counts, K, N, spare=1, seed=K + N)


@pytest.mark.parametrize("T,k,E,d,h", [
    (1, 1, 1, 8, 8), (1, 8, 128, 256, 128), (4, 8, 24, 2048, 768), (16, 4, 9, 136, 72), (100, 3, 7, 264, 40),
    (300, 2, 4, 520, 264), (1200, 2, 3, 768, 256), (2000, 4, 8, 512, 384), (640, 8, 64, 256, 96), (3000, 1, 2, 2880, 136),
    (900, 3, 3, 1032, 1000),
])
def test_up_swiglu(T, k, E, d, h):
    say(f"[gpu] mxfp4 gate/up T={T} k={k} E={E} d={d} h={h}")
    check_up(T, k, E, d, h, seed=T + d)


@pytest.mark.parametrize("T,k,E,d,h", [
    (1, 1, 1, 8, 8), (4, 8, 128, 256, 128), (16, 4, 9, 136, 72), (100, 3, 7, 264, 40), (60, 2, 4, 520, 1000),
    (1200, 2, 3, 768, 256), (2000, 4, 8, 512, 384), (900, 3, 3, 1032, 520), (700, 2, 5, 264, 8), (3000, 1, 2, 640, 776),
])
def test_up_swiglu_quantised(T, k, E, d, h):
    """The quantising launch writes what quantising the plain launch's rows gives, and nothing past M."""
    say(f"[gpu] mxfp4 gate/up to mxfp4 T={T} k={k} E={E} d={d} h={h}")
    rng = np.random.default_rng(T + h)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    x, _ = packed(rng, (T, d))
    w, _ = packed(rng, (E, 2 * h, d), 0.1)
    if T > 50:
        x.scales[T // 3, 0] = 255  # a NaN row stays one
    p = moe.moe_permute(torch.zeros((T, 8), dtype=torch.bfloat16, device=DEV), to_dev(ids), E, gather=False)
    M = int(p.offsets[-1])
    plain = moe.moe_gemm_up_swiglu_mxfp4(x, p.offsets, w, perm=p.perm, k=k)
    want = moe.moe_mxfp4_quantize(plain[:M].contiguous())
    q = torch.full((T * k, moe.mxfp4_row_bytes(h)), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((T * k, moe.mxfp4_scale_bytes(h)), 0xCD, dtype=torch.uint8, device=DEV)
    got = moe.moe_gemm_up_swiglu_mxfp4_q(x, p.offsets, w, perm=p.perm, k=k, q=q, scales=s)
    assert torch.equal(got.scales[:M], want.scales) and torch.equal(got.q[:M], want.q)
    assert (q[M:] == 0xAB).all() and (s[M:] == 0xCD).all(), "rows past M were written"


def test_up_swiglu_all_dropped_and_one_expert():
    say("[gpu] mxfp4 gate/up all dropped, one expert")
    check_up(50, 2, 5, 64, 32, ids=np.full((50, 2), -1, np.int32))
    check_up(400, 2, 5, 64, 32, ids=np.full((400, 2), 3, np.int32))
    check_up(900, 2, 2, 264, 136, ids=np.full((900, 2), 1, np.int32))


@pytest.mark.parametrize("rows", [40, 1200])
def test_products_with_large_gates_and_nan_blocks(rows):
    """Gates where exp overflows either way, and NaN blocks: only the rows and columns that hold them turn NaN."""
    say(f"[gpu] mxfp4 gate/up with large gates and NaN blocks, rows={rows}")
    rng = np.random.default_rng(1)
    K, h = 128, 64
    xv = np.full((rows, K), 4.0)
    wv = rng.normal(size=(1, 2 * h, K)) * 0.1
    wv[0, 0], wv[0, 1], wv[0, 2] = 6.0, -6.0, 0.0  # gates of 128 * 24 = 3e3, -3e3 and 0
    q, s = om.quantize(xv)
    s[1, 2] = 255
    x = moe.Mxfp4(to_dev(q), to_dev(s), K)
    wq, ws = om.quantize(wv[0])
    ws[h + 5, 0] = 255  # one up row
    w = moe.Mxfp4(to_dev(wq[None]), to_dev(ws[None]), K)
    offsets = to_dev(np.array([0, rows], dtype=np.int32))
    out = moe.moe_gemm_up_swiglu_mxfp4(x, offsets, w).float().cpu().numpy()
    assert np.isnan(out[1]).all() and np.isnan(out[:, 5]).all()
    keep = np.ones(rows, bool)
    keep[1] = False
    rest = np.delete(out[keep], 5, axis=1)
    assert np.isfinite(rest).all()
    assert (out[keep, 1] == 0).all() and (out[keep, 2] == 0).all() and (np.abs(out[keep, 0]) > 0).all()
    y = moe.moe_grouped_projection_mxfp4(x, offsets, w).float().cpu().numpy()
    assert np.isnan(y[1]).all() and np.isnan(y[:, h + 5]).all() and np.isfinite(np.delete(y[keep], h + 5, axis=1)).all()


@pytest.mark.parametrize("cap,offsets", [
    (50, [0, 60, 40, 90]), (50, [-5, 10, 20, 1000]), (50, [10, 5, 50, 50]), (1500, [0, 1600, 1400, 9000]),
    (1500, [700, 0, 1500, 1500]),
])
def test_offsets_outside_the_capacity(cap, offsets):
    """Offsets are clamped into the capacity: no row outside it is read or written."""
    say(f"[gpu] mxfp4 offsets {offsets} of {cap} rows")
    rng = np.random.default_rng(2)
    K, N, E = 72, 40, 3
    x, xv = packed(rng, (cap, K))
    w, wv = packed(rng, (E, N, K))
    buf = torch.full((cap + 64, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_projection_mxfp4(x, to_dev(np.array(offsets, dtype=np.int32)), w, y=buf[:cap])
    got = buf.double().cpu().numpy()
    assert (got[cap:] == 7.0).all()
    o = np.clip(offsets, 0, cap)
    owners = np.full(cap, -1)
    for e in range(E):
        owners[o[e]:max(o[e], o[e + 1])] = e
    for r in range(cap):
        if owners[r] >= 0 and sum(o[e] <= r < o[e + 1] for e in range(E)) == 1:
            want, tol = sums(xv[r:r + 1], wv[owners[r]])
            assert (np.abs(got[r] - want[0]) <= tol[0] + (np.abs(want[0]) + tol[0]) * 2.0 ** -8).all()
        elif owners[r] < 0:
            assert (got[r] == 7.0).all()


def test_whole_step_and_its_graph():
    """The step on MXFP4 experts is its calls one by one; captured, every replay equals the eager step."""
    say("[gpu] mxfp4 expert step")
    T, k, E, d, h = 300, 4, 9, 264, 136
    rng = np.random.default_rng(4)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[7] = -1
    ids, rw = to_dev(ids), to_dev(rng.random((T, k)).astype(np.float32))
    w_ug = moe.moe_mxfp4_quantize_weights(bf16(rng.normal(size=(E, 2 * h, d)) * 0.1).to(DEV), "out_in")
    w_down = moe.moe_mxfp4_quantize_weights(bf16(rng.normal(size=(E, h, d)) * 0.1).to(DEV), "in_out")
    x = bf16(rng.normal(size=(T, d))).to(DEV)
    y, p = moe.moe_expert_forward_mxfp4(x, ids, rw, w_ug, w_down)
    M = int(p.offsets[-1])
    xq = moe.moe_mxfp4_quantize(x)
    h_buf = moe.moe_gemm_up_swiglu_mxfp4(xq, p.offsets, w_ug, perm=p.perm, k=k)
    hq = moe.moe_mxfp4_quantize(h_buf)
    fused = moe.moe_gemm_up_swiglu_mxfp4_q(xq, p.offsets, w_ug, perm=p.perm, k=k)
    assert torch.equal(hq.q[:M], fused.q[:M]) and torch.equal(hq.scales[:M], fused.scales[:M])
    yp = moe.moe_grouped_projection_mxfp4(hq, p.offsets, w_down)
    assert torch.equal(moe.moe_unpermute(yp, p.inv_map, rw), y) and not y[7].any()
    # against 64 bits, from the quantised activations that the step itself made
    hv, wv = om.dequantize(hq.q.cpu().numpy(), hq.scales.cpu().numpy(), h), om.dequantize(w_down.q.cpu().numpy(), w_down.scales.cpu().numpy(), h)
    off = p.offsets.cpu().numpy()
    yv, ypv = np.zeros((T, d)), np.zeros((M, d))
    for e in range(E):
        ypv[off[e]:off[e + 1]] = hv[off[e]:off[e + 1]] @ wv[e].T
    inv = p.inv_map.cpu().numpy()
    mag = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                yv[t] += rw[t, j].item() * ypv[inv[t, j]]
                mag[t] += abs(rw[t, j].item()) * np.abs(ypv[inv[t, j]])
    # y_perm is rounded once to bf16 (2^-8), y once more; the fp32 sums are far below that here
    assert (np.abs(y.double().cpu().numpy() - yv) <= mag * 2.0 ** -8 * 1.01 + np.abs(yv) * 2.0 ** -8 * 1.01 + 1e-3 * mag).all()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        moe.moe_expert_forward_mxfp4(x, ids, rw, w_ug, w_down)
        with torch.cuda.graph(graph, stream=s):
            yg, _ = moe.moe_expert_forward_mxfp4(x, ids, rw, w_ug, w_down)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(3):
        x.copy_(bf16(rng.normal(size=(T, d))))
        want, _ = moe.moe_expert_forward_mxfp4(x, ids, rw, w_ug, w_down)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, want), rep


def test_no_rows():
    say("[gpu] mxfp4 products without rows")
    rng = np.random.default_rng(0)
    w, _ = packed(rng, (2, 16, 64))
    x = moe.Mxfp4(torch.empty((0, 32), dtype=torch.uint8, device=DEV), torch.empty((0, 16), dtype=torch.uint8, device=DEV), 64)
    z = to_dev(np.zeros(3, dtype=np.int32))
    assert moe.moe_grouped_projection_mxfp4(x, z, w).shape == (0, 16)
    assert moe.moe_gemm_up_swiglu_mxfp4(x, z, w, perm=torch.empty(0, dtype=torch.int32, device=DEV), k=4).shape == (0, 8)


def test_refusals():
    rng = np.random.default_rng(0)
    x, _ = packed(rng, (4, 64))
    w, _ = packed(rng, (2, 16, 64))
    off = to_dev(np.array([0, 2, 4], dtype=np.int32))
    with pytest.raises(ValueError):
        moe.moe_grouped_projection_mxfp4(x, off, moe.Mxfp4(w.q, w.scales, 32))
    with pytest.raises(ValueError):
        moe.moe_grouped_projection_mxfp4(x, off[:2], w)
    with pytest.raises(TypeError):
        moe.moe_grouped_projection_mxfp4(moe.Mxfp4(x.q.to(torch.int32), x.scales, 64), off, w)
    with pytest.raises(ValueError):
        moe.moe_gemm_up_swiglu_mxfp4(x, off, w, k=2)
    with pytest.raises(moe.MoeError, match="BAD_SHAPE"):
        moe.moe_mxfp4_quantize(torch.zeros((2, 12), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(moe.MoeError, match="MISALIGNED"):
        moe.moe_mxfp4_quantize(torch.zeros(2 * 16 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 16))
