"""Refusals and size arithmetic of the router and MXFP4 calls, on a host without a GPU (nothing is launched)."""

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

OK, NULLP, SHAPE, ALIGN, WS, DEV = range(6)
FAKE = 0x10000  # aligned, never dereferenced
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="valid sizes with placeholder pointers: host without a GPU only")


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def topk(lib, logits=FAKE, dtype=0, T=4, E=8, k=2, ids=FAKE, w=FAKE, lse=FAKE):
    return lib.moe_router_topk(logits, dtype, T, E, k, 1, ids, w, lse, None)


def losses(lib, logits=FAKE, dtype=0, T=4, E=8, k=2, ids=FAKE, w=FAKE, lse=FAKE, counts=FAKE, tokens=FAKE, mean=FAKE,
           out=FAKE, ws=FAKE, wsb=1 << 30):
    return lib.moe_router_topk_losses(logits, dtype, T, E, k, 1, ids, w, lse, counts, tokens, mean, out, ws, wsb, None)


def backward(lib, logits=FAKE, dtype=0, T=4, E=8, k=2, ids=FAKE, w=FAKE, counts=FAKE, tokens=FAKE, dw=FAKE, dl=FAKE,
             d=FAKE):
    return lib.moe_router_backward(logits, dtype, T, E, k, 1, ids, w, counts, tokens, dw, dl, d, None)


@pytest.mark.parametrize("fn", [topk, losses, backward])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), SHAPE), (dict(dtype=-1), SHAPE), (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(k=0), SHAPE), (dict(k=9), SHAPE), (dict(E=200, k=65), SHAPE), (dict(T=2**31, k=1), SHAPE),
    (dict(T=2**30, k=2), SHAPE), (dict(logits=None), NULLP), (dict(ids=None), NULLP), (dict(w=None), NULLP),
    (dict(logits=FAKE + 1), ALIGN), (dict(logits=FAKE + 2, dtype=1), ALIGN), (dict(ids=FAKE + 2), ALIGN),
    (dict(w=FAKE + 1), ALIGN),
])
def test_router_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(counts=None), NULLP), (dict(tokens=None), NULLP), (dict(mean=None), NULLP), (dict(out=None), NULLP),
    (dict(ws=None), NULLP), (dict(lse=None), NULLP), (dict(counts=FAKE + 2), ALIGN), (dict(ws=FAKE + 4), ALIGN),
    (dict(wsb=8), WS),
])
def test_router_losses_validation(lib, kw, status):
    assert losses(lib, **kw) == status


def test_router_backward_needs_what_its_gradients_use(lib):
    assert backward(lib, counts=None) == NULLP and backward(lib, tokens=None) == NULLP and backward(lib, d=None) == NULLP
    assert backward(lib, d=FAKE + 1) == ALIGN and backward(lib, dl=FAKE + 2) == ALIGN
    assert backward(lib, dl=None, counts=None, tokens=None) in (OK, DEV)
    assert backward(lib, dw=None, ids=None, w=None) in (OK, DEV)


@NO_GPU
def test_router_accepts(lib):
    for fn in (topk, losses, backward):
        assert fn(lib) == DEV
        assert fn(lib, logits=FAKE + 2) == DEV  # bf16 rows need no more than their own alignment
    assert topk(lib, T=0, logits=None, ids=None, w=None, lse=None) == DEV
    assert losses(lib, T=0, logits=None, ids=None, w=None, lse=None) == DEV


def test_router_workspace_bytes(lib):
    f = moe.router_workspace_bytes
    assert f(0, 64) == 132 * 4  # one workgroup's partial sums: 2 E + 2 words, in whole 16 bytes
    assert f(64, 64) == f(0, 64) and f(65, 64) == 2 * f(0, 64)
    assert f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 1025) == 0 and f(2**31, 4) == 0
    assert f(10**6, 64) == f(2**31 - 1, 64)  # bounded however many tokens


def test_mxfp4_sizes(lib):
    for K in (8, 24, 32, 40, 504, 512, 520, 2880):
        assert lib.moe_mxfp4_row_bytes(K) == moe.mxfp4_row_bytes(K) == 16 * -(-K // 32)
        assert lib.moe_mxfp4_scale_bytes(K) == moe.mxfp4_scale_bytes(K) == 16 * -(-K // 512)
    for K in (0, 4, 12, -8, (1 << 24) + 8):
        assert lib.moe_mxfp4_row_bytes(K) == 0 and lib.moe_mxfp4_scale_bytes(K) == 0


def quantize(lib, x=FAKE, rows=4, K=64, q=FAKE, s=FAKE):
    return lib.moe_mxfp4_quantize(x, rows, K, q, s, None)


def dequantize(lib, x=FAKE, rows=4, K=64, q=FAKE, s=FAKE):
    return lib.moe_mxfp4_dequantize(q, s, rows, K, x, None)


@pytest.mark.parametrize("fn", [quantize, dequantize])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=12), SHAPE), (dict(K=(1 << 24) + 8), SHAPE),
    (dict(rows=2**40, K=1 << 20), SHAPE), (dict(x=None), NULLP), (dict(q=None), NULLP), (dict(s=None), NULLP),
    (dict(x=FAKE + 8), ALIGN), (dict(q=FAKE + 4), ALIGN), (dict(s=FAKE + 8), ALIGN),
])
def test_mxfp4_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


def weights(lib, w=FAKE, layout=0, d_in=64, d_out=24, E=2, q=FAKE, s=FAKE):
    return lib.moe_mxfp4_quantize_weights(w, layout, d_in, d_out, E, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(layout=2), SHAPE), (dict(d_in=4), SHAPE), (dict(d_out=12), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(d_in=(1 << 20) + 8), SHAPE), (dict(w=None), NULLP), (dict(q=None), NULLP), (dict(s=None), NULLP),
    (dict(w=FAKE + 2), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(s=FAKE + 1), ALIGN),
])
def test_mxfp4_weights_validation(lib, kw, status):
    assert weights(lib, **kw) == status


def projection(lib, xq=FAKE, xs=FAKE, offs=FAKE, wq=FAKE, ws=FAKE, cap=16, d_in=64, d_out=24, E=2, out=FAKE):
    return lib.moe_grouped_projection_mxfp4(xq, xs, offs, wq, ws, cap, d_in, d_out, E, out, None)


def up(lib, xq=FAKE, xs=FAKE, offs=FAKE, wq=FAKE, ws=FAKE, cap=16, d_in=64, d_out=24, E=2, out=FAKE, perm=FAKE, k=2):
    return lib.moe_gemm_up_swiglu_mxfp4(xq, xs, perm, cap, k, offs, wq, ws, d_in, d_out, E, out, None)


def up_q(lib, xq=FAKE, xs=FAKE, offs=FAKE, wq=FAKE, ws=FAKE, cap=16, d_in=64, d_out=24, E=2, out=FAKE, perm=FAKE, k=2,
         out_s=FAKE):
    return lib.moe_gemm_up_swiglu_mxfp4_q(xq, xs, perm, cap, k, offs, wq, ws, d_in, d_out, E, out, out_s, None)


@pytest.mark.parametrize("fn", [projection, up, up_q])
@pytest.mark.parametrize("kw,status", [
    (dict(cap=-1), SHAPE), (dict(d_in=12), SHAPE), (dict(d_out=4), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(d_in=(1 << 20) + 8), SHAPE), (dict(d_out=(1 << 20) + 8), SHAPE), (dict(cap=2**31), SHAPE),
    (dict(xq=None), NULLP), (dict(xs=None), NULLP), (dict(offs=None), NULLP), (dict(wq=None), NULLP),
    (dict(ws=None), NULLP), (dict(out=None), NULLP), (dict(xq=FAKE + 8), ALIGN), (dict(xs=FAKE + 4), ALIGN),
    (dict(wq=FAKE + 8), ALIGN), (dict(ws=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN), (dict(offs=FAKE + 2), ALIGN),
])
def test_mxfp4_product_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


def test_mxfp4_up_gather_validation(lib):
    assert up(lib, k=0) == SHAPE and up(lib, cap=2**30, k=2) == SHAPE and up(lib, perm=FAKE + 2) == ALIGN
    assert up(lib, perm=None, k=2) == SHAPE  # sorted rows are taken one by one
    assert up(lib, perm=None, k=1) in (OK, DEV)
    assert up_q(lib, out_s=None) == NULLP and up_q(lib, out_s=FAKE + 8) == ALIGN and up_q(lib, perm=None, k=2) == SHAPE
    assert projection(lib, cap=0, xq=None, xs=None, out=None) in (OK, DEV)
    assert up_q(lib, cap=0, xq=None, xs=None, out=None, out_s=None) in (OK, DEV)


def test_binding_refusals_without_a_gpu():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    for bad in (x.half(), x.to(torch.int32)):
        with pytest.raises(TypeError):
            moe.moe_router_topk(bad, 2)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x, 2)  # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_router_topk(x[0], 2)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize(x)
    with pytest.raises(TypeError):
        moe.moe_mxfp4_dequantize(x)
    m = moe.Mxfp4(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.uint8), 8)
    with pytest.raises(ValueError):
        moe.moe_grouped_projection_mxfp4(m, torch.zeros(2, dtype=torch.int32), m)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize_weights(x[None], "io")
