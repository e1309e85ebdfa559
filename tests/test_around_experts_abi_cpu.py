"""Refusals and size arithmetic of the norms, AdamW and the 4-bit experts, on a host without a GPU (nothing is launched)."""

import ctypes
import math

import pytest
import torch

import ragged_grouped_gemm_histogram_amd as moe

OK, NULLP, SHAPE, ALIGN, WS, DEV, VALUE = 0, 1, 2, 3, 4, 5, 8
F = 0x10000  # aligned, never dereferenced
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: host without a GPU only")


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def test_status_string(lib):
    assert lib.moe_status_string(VALUE).decode().startswith("MOE_ERR_BAD_VALUE")


# ---------------------------------------------------------------- norms


def before(lib, x=F, xt=0, w=F, wt=0, eps=1e-6, T=4, d=64, y=F):
    return lib.moe_rmsnorm(x, xt, w, wt, eps, T, d, y, None)


def before_back(lib, dy=F, more=F, x=F, xt=0, w=F, wt=0, eps=1e-6, add=F, T=4, d=64, y=F, dw=F, ws=F, wsb=1 << 30):
    return lib.moe_rmsnorm_backward(dy, more, x, xt, w, wt, eps, add, T, d, y, dw, ws, wsb, None)


def after(lib, b=F, x=F, xt=0, flags=3, wp=F, w=F, wt=0, gate=F, kind=2, a=1.0, s=1.0, eps=1e-6, T=4, d=64, y=F, n=F):
    return lib.moe_residual_norm(b, x, xt, flags, wp, w, wt, gate, kind, a, s, eps, T, d, y, n, None)


def after_back(lib, dr=F, dn=F, more=F, b=F, x=F, xt=0, flags=3, wp=F, w=F, wt=0, gate=F, kind=2, a=1.0, s=1.0, eps=1e-6,
               T=4, d=64, y=F, dy=F, dg=F, dwp=F, dw=F, ws=F, wsb=1 << 30):
    return lib.moe_residual_norm_backward(dr, dn, more, b, x, xt, flags, wp, w, wt, gate, kind, a, s, eps, T, d, y, dy, dg,
                                          dwp, dw, ws, wsb, None)


@pytest.mark.parametrize("fn", [before, before_back, after, after_back])
@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), SHAPE), (dict(xt=-1), SHAPE), (dict(wt=2), SHAPE), (dict(T=-1), SHAPE), (dict(T=2**31), SHAPE),
    (dict(d=0), SHAPE), (dict(d=12), SHAPE), (dict(d=-8), SHAPE), (dict(d=16392), SHAPE), (dict(eps=-1e-9), VALUE),
    (dict(eps=math.nan), VALUE), (dict(eps=math.inf), VALUE), (dict(x=None), NULLP), (dict(y=None), NULLP),
    (dict(x=F + 8), ALIGN), (dict(y=F + 2), ALIGN), (dict(w=F + 4), ALIGN),
])
def test_norm_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


@pytest.mark.parametrize("fn", [after, after_back])
@pytest.mark.parametrize("kw,status", [
    (dict(flags=4), SHAPE), (dict(flags=-1), SHAPE), (dict(kind=3), SHAPE), (dict(kind=-1), SHAPE),
    (dict(a=math.inf), VALUE), (dict(s=math.nan), VALUE), (dict(b=None), NULLP), (dict(gate=None), NULLP),
    (dict(gate=None, kind=1), NULLP), (dict(b=F + 8), ALIGN), (dict(wp=F + 8), ALIGN), (dict(gate=F + 8), ALIGN),
    (dict(gate=F + 2, kind=1), ALIGN),
])
def test_residual_norm_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


def test_norm_takes_what_its_flags_need(lib):
    assert after(lib, n=None) == NULLP and after(lib, n=F + 8) == ALIGN
    assert after(lib, flags=1, n=None, w=None) == DEV and after(lib, kind=0, gate=None) == DEV
    assert after(lib, kind=1, gate=F + 4) == DEV and after(lib, wp=None, w=None) == DEV
    assert before(lib, w=None) == DEV and before(lib, T=0, x=None, y=None) == DEV
    assert before_back(lib, dy=None) == NULLP and before_back(lib, more=F + 8) == ALIGN
    assert before_back(lib, more=None, add=None, dw=None, w=None) == DEV
    assert before_back(lib, ws=None) == NULLP and before_back(lib, ws=F + 8) == ALIGN and before_back(lib, wsb=8) == WS
    assert before_back(lib, T=0, dy=None, more=None, x=None, add=None, y=None, ws=None, wsb=0) == DEV
    assert after_back(lib, dr=None) == DEV and after_back(lib, dr=None, flags=1) == NULLP
    assert after_back(lib, dn=None) == NULLP and after_back(lib, dn=None, x=None, flags=1) == DEV
    assert after_back(lib, b=None, flags=2, kind=0, gate=None, dg=None) == DEV
    assert after_back(lib, dg=None) == NULLP and after_back(lib, dy=None) == NULLP
    assert after_back(lib, dwp=None, dw=None) == DEV and after_back(lib, dg=F + 2) == ALIGN
    assert after_back(lib, wsb=8) == WS and after_back(lib, ws=None) == NULLP and after_back(lib, more=F + 2) == ALIGN


def test_norm_workspace_bytes(lib):
    f = moe.norm_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 12) == 0 and f(4, 16392) == 0
    assert f(1, 64) == 64 * 12 and f(1, 16384) == 16384 * 12  # one row of three sums
    assert f(2**31 - 1, 64) == f(10**6, 64)  # bounded however many rows


# ---------------------------------------------------------------- AdamW


def tensors(*rows):
    table = (moe._AdamTensor * max(1, len(rows)))()
    for t, r in zip(table, rows):
        t.n, t.offset, t.param_dtype, t.grad_dtype = r[2:]
    return table


def addresses(rows, at):
    return (ctypes.c_void_p * max(1, len(rows)))(*[r[at] for r in rows])


def adamw(lib, rows=((F, F, 40, 0, 0, 1), (F, F, 3, 64, 1, 0)), count=None, bits=32, length=96, m=F, ms=F, v=F, vs=F, master=F,
          lr_ptr=None, step_ptr=None, scale=None, hyper=True, lists=True, **kw):
    h = moe._AdamHyper(1e-3, 0.9, 0.999, 1e-8, 0.1, 1, 0, 0)
    for k, val in kw.items():
        setattr(h, k, val)
    table, params, grads = tensors(*rows), addresses(rows, 0), addresses(rows, 1)
    return lib.moe_adamw_step(*(ctypes.addressof(a) if lists else None for a in (table, params, grads)),
                              len(rows) if count is None else count, bits, length, m, ms, v, vs, master,
                              ctypes.addressof(h) if hyper else None, lr_ptr, step_ptr, scale, None)


A = (F, F, 40, 0, 0, 1)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), SHAPE), (dict(bits=16), SHAPE), (dict(bits=0), SHAPE), (dict(length=-32), SHAPE),
    (dict(length=100), SHAPE), (dict(length=64), SHAPE), (dict(hyper=False), NULLP), (dict(lists=False), NULLP), (dict(m=None), NULLP),
    (dict(v=None), NULLP), (dict(bits=8, ms=None), NULLP), (dict(bits=8, vs=None), NULLP), (dict(m=F + 8), ALIGN),
    (dict(v=F + 4), ALIGN), (dict(master=F + 8), ALIGN), (dict(lr_ptr=F + 2), ALIGN), (dict(step_ptr=F + 1), ALIGN),
    (dict(scale=F + 2), ALIGN), (dict(rows=((F, F, 40, 0, 2, 0),)), SHAPE), (dict(rows=((F, F, 40, 0, 0, -1),)), SHAPE),
    (dict(rows=((F, F, -1, 0, 0, 0),)), SHAPE), (dict(rows=((F, F, 4, 8, 0, 0),)), SHAPE),
    (dict(rows=((F, F, 4, -32, 0, 0),)), SHAPE), (dict(rows=((F, F, 2**40, 0, 0, 0),)), SHAPE),
    (dict(rows=((F, F, 1, 128, 0, 0),)), SHAPE), (dict(rows=(A, A)), SHAPE), (dict(rows=(A, (F, F, 1, 32, 0, 0))), SHAPE),
    (dict(rows=((None, F, 4, 0, 0, 0),)), NULLP), (dict(rows=((F, None, 4, 0, 0, 0),)), NULLP),
    (dict(rows=((F + 1, F, 4, 0, 0, 0),)), ALIGN), (dict(rows=((F, F + 2, 4, 0, 0, 1),)), ALIGN),
    (dict(lr=math.inf), VALUE), (dict(lr=math.nan), VALUE), (dict(beta1=1.0), VALUE), (dict(beta1=-0.1), VALUE),
    (dict(beta2=1.0), VALUE), (dict(beta2=math.nan), VALUE), (dict(eps=-1.0), VALUE), (dict(eps=math.inf), VALUE),
    (dict(weight_decay=-0.1), VALUE), (dict(step=0), VALUE), (dict(step=2**31), VALUE),
])
def test_adamw_validation(lib, kw, status):
    assert adamw(lib, **kw) == status


def test_adamw_accepts(lib):
    assert adamw(lib) == DEV and adamw(lib, bits=8) == DEV and adamw(lib, ms=None, vs=None, master=None) == DEV
    assert adamw(lib, rows=((F + 2, F + 4, 4, 0, 0, 1),)) == DEV  # values need no more than their own alignment
    assert adamw(lib, rows=((None, None, 0, 0, 0, 0), A)) == DEV and adamw(lib, rows=()) == DEV
    assert adamw(lib, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0) == DEV


def moments(lib, m=F, ms=F, v=F, vs=F, n=64, mo=F, vo=F):
    return lib.moe_adamw_moments(m, ms, v, vs, n, mo, vo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-32), SHAPE), (dict(n=40), SHAPE), (dict(m=None), NULLP), (dict(ms=None), NULLP), (dict(v=None), NULLP),
    (dict(vs=None), NULLP), (dict(mo=None), NULLP), (dict(vo=None), NULLP), (dict(m=F + 4), ALIGN), (dict(vo=F + 8), ALIGN),
    (dict(n=0, m=None, ms=None, v=None, vs=None, mo=None, vo=None), DEV),
])
def test_adamw_moments_validation(lib, kw, status):
    assert moments(lib, **kw) == status


# ---------------------------------------------------------------- 4-bit experts


def quantize(lib, w=F, layout=0, d_in=64, d_out=24, E=2, group=32, q=F, s=F, z=F):
    return lib.moe_int4_quantize_weights(w, layout, d_in, d_out, E, group, q, s, z, None)


def dequantize(lib, w=F, d_in=64, d_out=24, E=2, group=32, q=F, s=F, z=F):
    return lib.moe_int4_dequantize_weights(q, s, z, d_in, d_out, E, group, w, None)


def projection(lib, x=F, offs=F, q=F, s=F, z=F, group=32, cap=16, d_in=64, d_out=24, E=2, w=F):
    return lib.moe_grouped_projection_int4(x, offs, q, s, z, group, cap, d_in, d_out, E, w, None)


def up(lib, x=F, offs=F, q=F, s=F, z=F, group=32, cap=16, d_in=64, d_out=24, E=2, w=F, perm=F, k=2):
    return lib.moe_gemm_up_swiglu_int4(x, perm, cap, k, offs, q, s, z, group, d_in, d_out, E, w, None)


@pytest.mark.parametrize("fn", [quantize, dequantize, projection, up])
@pytest.mark.parametrize("kw,status", [
    (dict(group=16), SHAPE), (dict(group=0), SHAPE), (dict(group=256), SHAPE), (dict(d_in=12), SHAPE),
    (dict(d_out=4), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(d_in=(1 << 20) + 8), SHAPE),
    (dict(w=None), NULLP), (dict(q=None), NULLP), (dict(s=None), NULLP), (dict(w=F + 2), ALIGN), (dict(q=F + 8), ALIGN),
    (dict(s=F + 8), ALIGN), (dict(z=F + 4), ALIGN), (dict(z=None), DEV), (dict(z=F + 8), DEV),
])
def test_int4_validation(lib, fn, kw, status):
    assert fn(lib, **kw) == status


def test_int4_products_validation(lib):
    for fn in (projection, up):
        assert fn(lib, cap=-1) == SHAPE and fn(lib, x=None) == NULLP and fn(lib, offs=None) == NULLP
        assert fn(lib, x=F + 8) == ALIGN and fn(lib, offs=F + 2) == ALIGN and fn(lib, cap=0, x=None, w=None) == DEV
    assert up(lib, k=0) == SHAPE and up(lib, cap=2**30, k=2) == SHAPE and up(lib, perm=F + 2) == ALIGN
    assert up(lib, perm=None, k=2) == SHAPE and up(lib, perm=None, k=1) == DEV and projection(lib, cap=2**31) == SHAPE
    assert quantize(lib, layout=2) == SHAPE


# ---------------------------------------------------------------- the binding


def test_binding_refuses_on_the_cpu():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64)
    for bad in (x.half(), x.to(torch.int32)):
        with pytest.raises(TypeError):
            moe.moe_rmsnorm(bad, w)
    for call in (lambda: moe.moe_rmsnorm(x, w), lambda: moe.moe_rmsnorm(x[0], w), lambda: moe.moe_residual_norm(x, x),
                 lambda: moe.moe_residual_norm_backward(x, x, x, x), lambda: moe.moe_rmsnorm_backward(x, x, w),
                 lambda: moe.moe_int4_quantize_weights(x[None], group=32), lambda: moe.moe_adamw_state([x]),
                 lambda: moe.moe_adamw_state([]), lambda: moe.moe_adamw_state([x], bits=16),
                 lambda: moe.moe_int4_quantize_weights(x[None], "io")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.moe_int4_dequantize_weights(x)
    with pytest.raises(TypeError):
        moe.moe_grouped_projection_int4(x, torch.zeros(3, dtype=torch.int32), x)
