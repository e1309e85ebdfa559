"""Python binding of libmoe_grouped, the routed MoE expert step on MI355X (gfx950).

Argument marshalling only: every step runs in the HIP library's kernels. torch
supplies device memory and the current stream. The functions mirror the C ABI
declared in ``include/moe_grouped.h``; the optional ``out=`` tensors let a
caller keep fixed capacity-shaped buffers across calls.

The library must have been built (``python -m ragged_grouped_gemm_histogram_amd.build``);
every call raises ImportError when it is missing. There is no other code path.
"""

from __future__ import annotations

import ctypes
import functools
import os
import re
from dataclasses import dataclass, field

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_grouped.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_grouped.h")
MAX_EXPERTS = 1024

MOE_OK = 0

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_f32 = ctypes.c_float
_SIGNATURES = {
    "moe_permute_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "moe_permute": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_permute_noalloc": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "grouped_swiglu_expert": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp]),
    "moe_gemm_up_swiglu": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_gemm_up_swiglu_u": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp]),
    "moe_gemm_down": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_gemm_up_swiglu_gather": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "grouped_swiglu_expert_gather": (ctypes.c_int,
                                     [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "moe_unpermute": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i64, _vp, _vp]),
    "moe_grouped_projection": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_swiglu_backward": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp]),
    "moe_grouped_dgrad": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_grouped_wgrad_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "moe_grouped_wgrad": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _sz, _vp]),
    "moe_permute_backward": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i64, _vp, _vp]),
    "moe_unpermute_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i64, _vp, _vp, _vp]),
    "moe_router_workspace_bytes": (_sz, [_i64, _i32]),
    "moe_router_topk": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "moe_router_topk_losses": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _sz, _vp]),
    "moe_router_backward": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_mxfp4_row_bytes": (_sz, [_i64]),
    "moe_mxfp4_scale_bytes": (_sz, [_i64]),
    "moe_mxfp4_quantize": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "moe_mxfp4_quantize_weights": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp]),
    "moe_mxfp4_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "moe_grouped_projection_mxfp4": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_gemm_up_swiglu_mxfp4": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "moe_gemm_up_swiglu_mxfp4_q": (ctypes.c_int,
                                   [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "moe_rmsnorm": (ctypes.c_int, [_vp, _i32, _vp, _i32, _f32, _i64, _i64, _vp, _vp]),
    "moe_residual_norm": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _f32, _f32, _f32, _i64, _i64,
                                         _vp, _vp, _vp]),
    "moe_norm_workspace_bytes": (_sz, [_i64, _i64]),
    "moe_rmsnorm_backward": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _i32, _f32, _vp, _i64, _i64, _vp, _vp, _vp, _sz,
                                            _vp]),
    "moe_residual_norm_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _f32, _f32,
                                                  _f32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_adamw_step": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_adamw_moments": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
    "moe_int4_quantize_weights": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp]),
    "moe_int4_dequantize_weights": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp]),
    "moe_grouped_projection_int4": (ctypes.c_int,
                                    [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp]),
    "moe_gemm_up_swiglu_int4": (ctypes.c_int,
                                [_vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _vp, _vp]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}

W_LAYOUTS = {"in_out": 0, "out_in": 1}  # [E, d_in, d_out] / [E, d_out, d_in]


_LIB = None


def load_library() -> ctypes.CDLL:
    """Load libmoe_grouped.so (once). Raises ImportError when it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m ragged_grouped_gemm_histogram_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {load_library().moe_status_string(status).decode()}")


def header_functions() -> list[str]:
    """Names of the functions declared in include/moe_grouped.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return re.findall(r"^\s*(?:moe_status|size_t|const char\*)\s+(\w+)\s*\(", text, flags=re.M)


def _check(status: int, call: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, call)


def _public_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# Names that every call looks up, bound once. The two device queries are those behind torch.cuda.current_device() and
# current_stream(), two microseconds a call less; a torch that lacks them (one without a GPU backend) has the public ones.
_Tensor = torch.Tensor
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)


def _stream(t: torch.Tensor) -> int:
    # The library launches on the current HIP device; a stream of another device would fail the launch.
    index = t.get_device()
    if index != _current_device():
        raise ValueError(f"tensors are on {t.device} but the current device is cuda:{torch.cuda.current_device()}; "
                         "call inside torch.cuda.device(...)")
    return _raw_stream(index)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()  # 0, NULL to the library, without elements


def _want(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device) -> torch.Tensor:
    # (one device index compared instead of device objects: a CPU tensor's is -1, a CPU device's None)
    if (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == device.index
            and t.is_contiguous()):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or t.device.type != "cuda":
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == device.index
            and t.is_contiguous()):
        return t
    return _want(t, name, dtype, shape, device)


@dataclass
class Permuted:
    x_perm: torch.Tensor  # bf16 [T*k, d]; rows [0, M) valid
    counts: torch.Tensor  # int32 [E]
    offsets: torch.Tensor  # int32 [E+1]
    perm: torch.Tensor  # int32 [T*k]; entries [0, M) valid
    inv_map: torch.Tensor  # int32 [T, k]; -1 for dropped slots


def permute_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(load_library().moe_permute_workspace_bytes(T, k, E))


def moe_permute(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int, *, x_perm=None, counts=None,
                offsets=None, perm=None, inv_map=None, workspace=None, gather: bool = True) -> Permuted:
    """Histogram, offsets, stable order, inverse map and permuted gather (one stream, no sync).

    ``gather=False`` skips the row copy (``x_perm`` is None); a ``*_gather`` GEMM then reads X through perm.
    """
    if x.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("x must be [T, d] and expert_ids [T, k]")
    T, d = x.shape
    k = expert_ids.shape[1]
    dev = x.device
    _want(x, "x", torch.bfloat16, (T, d), dev)
    _want(expert_ids, "expert_ids", torch.int32, (T, k), dev)
    S = T * k
    E = int(num_experts)
    x_perm = _out(x_perm, "x_perm", torch.bfloat16, (S, d), dev) if gather else None
    counts = _out(counts, "counts", torch.int32, (E,), dev)
    offsets = _out(offsets, "offsets", torch.int32, (E + 1,), dev)
    perm = _out(perm, "perm", torch.int32, (S,), dev)
    inv_map = _out(inv_map, "inv_map", torch.int32, (T, k), dev)
    need = permute_workspace_bytes(T, k, E)
    if workspace is None:
        workspace = torch.empty((max(need, 4),), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    _check(load_library().moe_permute(_ptr(x) if gather else None, _ptr(expert_ids), T, k, d, E, _ptr(x_perm),
                                      _ptr(counts), _ptr(offsets),
                           _ptr(perm), _ptr(inv_map), _ptr(workspace), workspace.numel(), _stream(x)),
           "moe_permute")
    return Permuted(x_perm, counts, offsets, perm, inv_map)


def moe_permute_noalloc(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int, *, x_perm: torch.Tensor | None,
                        counts: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor,
                        inv_map: torch.Tensor) -> Permuted:
    """moe_permute without a workspace, for callers that cannot allocate: the histogram table is the library's
    fixed per-device array (at most ``E * ceil(T*k/256) <= 2**20`` entries). Every output is the caller's own
    tensor, so this call allocates nothing; ``x_perm=None`` skips the row copy. Calls that overlap on one GPU
    share the table and race."""
    if x.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("x must be [T, d] and expert_ids [T, k]")
    T, d = x.shape
    k = expert_ids.shape[1]
    dev = x.device
    _want(x, "x", torch.bfloat16, (T, d), dev)
    _want(expert_ids, "expert_ids", torch.int32, (T, k), dev)
    S, E = T * k, int(num_experts)
    if x_perm is not None:
        _want(x_perm, "x_perm", torch.bfloat16, (S, d), dev)
    _want(counts, "counts", torch.int32, (E,), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(perm, "perm", torch.int32, (S,), dev)
    _want(inv_map, "inv_map", torch.int32, (T, k), dev)
    _check(load_library().moe_permute_noalloc(_ptr(x) if x_perm is not None else None, _ptr(expert_ids), T, k, d,
                                              E, _ptr(x_perm), _ptr(counts), _ptr(offsets), _ptr(perm),
                                              _ptr(inv_map), _stream(x)), "moe_permute_noalloc")
    return Permuted(x_perm, counts, offsets, perm, inv_map)


def _gemm_shapes(a: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor):
    if a.dim() != 2 or w.dim() != 3 or offsets.dim() != 1:
        raise ValueError("expected a 2-D activation buffer, 1-D offsets and 3-D expert weights")
    return a.shape[0], a.device


def moe_gemm_up_swiglu(x_perm: torch.Tensor, offsets: torch.Tensor, w_ug: torch.Tensor, *, h_buf=None) -> torch.Tensor:
    """h_buf[rows_e] = bf16(SiLU(bf16(G)) * bf16(U)), [G|U] = x_perm[rows_e] @ W_ug[e]^T (one launch)."""
    cap, dev = _gemm_shapes(x_perm, offsets, w_ug)
    E, two_h, d = w_ug.shape
    h = two_h // 2
    _want(x_perm, "x_perm", torch.bfloat16, (cap, d), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_ug, "w_ug", torch.bfloat16, (E, 2 * h, d), dev)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (cap, h), dev)
    _check(load_library().moe_gemm_up_swiglu(_ptr(x_perm), _ptr(offsets), _ptr(w_ug), cap, d, h, E, _ptr(h_buf),
                                  _stream(x_perm)), "moe_gemm_up_swiglu")
    return h_buf


def moe_gemm_up_swiglu_u(x_perm: torch.Tensor, offsets: torch.Tensor, w_ug: torch.Tensor, *, h_buf=None,
                         u_buf=None) -> tuple[torch.Tensor, torch.Tensor]:
    """moe_gemm_up_swiglu that also stores the pre-activation u_buf = [G | U] = bf16(x_perm[rows_e] @ W_ug[e]^T)
    ([cap, 2h], gate block first) for the backward; returns (h_buf, u_buf). One launch."""
    cap, dev = _gemm_shapes(x_perm, offsets, w_ug)
    E, two_h, d = w_ug.shape
    h = two_h // 2
    _want(x_perm, "x_perm", torch.bfloat16, (cap, d), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_ug, "w_ug", torch.bfloat16, (E, 2 * h, d), dev)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (cap, h), dev)
    u_buf = _out(u_buf, "u_buf", torch.bfloat16, (cap, 2 * h), dev)
    _check(load_library().moe_gemm_up_swiglu_u(_ptr(x_perm), _ptr(offsets), _ptr(w_ug), cap, d, h, E, _ptr(h_buf),
                                               _ptr(u_buf), _stream(x_perm)), "moe_gemm_up_swiglu_u")
    return h_buf, u_buf


def moe_gemm_up_swiglu_gather(x: torch.Tensor, perm: torch.Tensor, offsets: torch.Tensor, w_ug: torch.Tensor,
                              k: int, *, h_buf=None) -> torch.Tensor:
    """moe_gemm_up_swiglu on token rows gathered through perm: sorted row p reads x[perm[p] // k] (one launch)."""
    if x.dim() != 2 or w_ug.dim() != 3:
        raise ValueError("expected x [T, d] and w_ug [E, 2h, d]")
    T, d = x.shape
    E, two_h, _ = w_ug.shape
    h = two_h // 2
    S = T * int(k)
    dev = x.device
    _want(x, "x", torch.bfloat16, (T, d), dev)
    _want(perm, "perm", torch.int32, (S,), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_ug, "w_ug", torch.bfloat16, (E, 2 * h, d), dev)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (S, h), dev)
    _check(load_library().moe_gemm_up_swiglu_gather(_ptr(x), _ptr(perm), T, int(k), _ptr(offsets), _ptr(w_ug), d, h,
                                                    E, _ptr(h_buf), _stream(x)), "moe_gemm_up_swiglu_gather")
    return h_buf


def grouped_swiglu_expert_gather(x: torch.Tensor, perm: torch.Tensor, offsets: torch.Tensor, w_ug: torch.Tensor,
                                 w_down: torch.Tensor, k: int, *, h_buf=None, y_perm=None):
    """grouped_swiglu_expert with the permuted gather fused into the gate/up loads: returns (h_buf, y_perm)."""
    if x.dim() != 2 or w_ug.dim() != 3 or w_down.dim() != 3:
        raise ValueError("expected x [T, d], w_ug [E, 2h, d], w_down [E, h, d]")
    T, d = x.shape
    E, two_h, _ = w_ug.shape
    h = two_h // 2
    S = T * int(k)
    dev = x.device
    _want(x, "x", torch.bfloat16, (T, d), dev)
    _want(perm, "perm", torch.int32, (S,), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_ug, "w_ug", torch.bfloat16, (E, 2 * h, d), dev)
    _want(w_down, "w_down", torch.bfloat16, (E, h, d), dev)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (S, h), dev)
    y_perm = _out(y_perm, "y_perm", torch.bfloat16, (S, d), dev)
    _check(load_library().grouped_swiglu_expert_gather(_ptr(x), _ptr(perm), T, int(k), _ptr(offsets), _ptr(w_ug),
                                                       _ptr(w_down), d, h, E, _ptr(h_buf), _ptr(y_perm), _stream(x)),
           "grouped_swiglu_expert_gather")
    return h_buf, y_perm


def moe_gemm_down(h_buf: torch.Tensor, offsets: torch.Tensor, w_down: torch.Tensor, *, y_perm=None) -> torch.Tensor:
    """y_perm[rows_e] = bf16(h_buf[rows_e] @ W_down[e]) (one launch)."""
    cap, dev = _gemm_shapes(h_buf, offsets, w_down)
    E, h, d = w_down.shape
    _want(h_buf, "h_buf", torch.bfloat16, (cap, h), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_down, "w_down", torch.bfloat16, (E, h, d), dev)
    y_perm = _out(y_perm, "y_perm", torch.bfloat16, (cap, d), dev)
    _check(load_library().moe_gemm_down(_ptr(h_buf), _ptr(offsets), _ptr(w_down), cap, d, h, E, _ptr(y_perm), _stream(h_buf)),
           "moe_gemm_down")
    return y_perm


def grouped_swiglu_expert(x_perm: torch.Tensor, offsets: torch.Tensor, w_ug: torch.Tensor, w_down: torch.Tensor, *,
                          h_buf=None, y_perm=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Eq 13 for every expert's row block: returns (h_buf, y_perm), both [cap, *] with rows [0, M) valid."""
    cap, dev = _gemm_shapes(x_perm, offsets, w_ug)
    E, two_h, d = w_ug.shape
    h = two_h // 2
    _want(x_perm, "x_perm", torch.bfloat16, (cap, d), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w_ug, "w_ug", torch.bfloat16, (E, 2 * h, d), dev)
    _want(w_down, "w_down", torch.bfloat16, (E, h, d), dev)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (cap, h), dev)
    y_perm = _out(y_perm, "y_perm", torch.bfloat16, (cap, d), dev)
    _check(load_library().grouped_swiglu_expert(_ptr(x_perm), _ptr(offsets), _ptr(w_ug), _ptr(w_down), cap, d, h, E,
                                     _ptr(h_buf), _ptr(y_perm), _stream(x_perm)), "grouped_swiglu_expert")
    return h_buf, y_perm


def moe_unpermute(y_perm: torch.Tensor, inv_map: torch.Tensor, routing_w: torch.Tensor, *, y=None) -> torch.Tensor:
    """y[t] = bf16(sum_j w[t,j] * y_perm[inv_map[t,j]]) over kept slots (atomic-free gather + reduce)."""
    if inv_map.dim() != 2:
        raise ValueError("inv_map must be [T, k]")
    T, k = inv_map.shape
    dev = y_perm.device
    d = y_perm.shape[1]
    _want(y_perm, "y_perm", torch.bfloat16, (T * k, d), dev)
    _want(inv_map, "inv_map", torch.int32, (T, k), dev)
    _want(routing_w, "routing_w", torch.float32, (T, k), dev)
    y = _out(y, "y", torch.bfloat16, (T, d), dev)
    _check(load_library().moe_unpermute(_ptr(y_perm), _ptr(inv_map), _ptr(routing_w), T, k, d, _ptr(y), _stream(y_perm)),
           "moe_unpermute")
    return y


def _w_dims(w: torch.Tensor, layout: str):
    if layout not in W_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(W_LAYOUTS)}, got {layout!r}")
    if w.dim() != 3:
        raise ValueError("expert weights must be 3-D")
    E, a, b = w.shape
    return (E, a, b) if layout == "in_out" else (E, b, a)  # E, d_in, d_out


def moe_grouped_projection(x: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor, layout: str = "in_out", *,
                           y=None) -> torch.Tensor:
    """Y[rows_e] = bf16(X[rows_e] @ W_e) with W_e [d_in, d_out] stored per ``layout`` (one launch)."""
    E, d_in, d_out = _w_dims(w, layout)
    if x.dim() != 2:
        raise ValueError("x must be [cap_rows, d_in]")
    cap, dev = x.shape[0], x.device
    _want(x, "x", torch.bfloat16, (cap, d_in), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w, "w", torch.bfloat16, tuple(w.shape), dev)
    y = _out(y, "y", torch.bfloat16, (cap, d_out), dev)
    _check(load_library().moe_grouped_projection(_ptr(x), _ptr(offsets), _ptr(w), W_LAYOUTS[layout], cap, d_in, d_out,
                                                 E, _ptr(y), _stream(x)), "moe_grouped_projection")
    return y


def moe_swiglu_backward(dh: torch.Tensor, u: torch.Tensor, offsets: torch.Tensor, *, du=None) -> torch.Tensor:
    """dU = [dG | dUp] of H = SiLU(G) * Up over the sorted rows [0, offsets[E]) (one launch)."""
    if dh.dim() != 2 or u.dim() != 2 or offsets.dim() != 1:
        raise ValueError("expected dh [cap, h], u [cap, 2h] and offsets [E+1]")
    cap, h = dh.shape
    E = offsets.shape[0] - 1
    dev = dh.device
    _want(dh, "dh", torch.bfloat16, (cap, h), dev)
    _want(u, "u", torch.bfloat16, (cap, 2 * h), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    du = _out(du, "du", torch.bfloat16, (cap, 2 * h), dev)
    _check(load_library().moe_swiglu_backward(_ptr(dh), _ptr(u), _ptr(offsets), E, cap, h, _ptr(du), _stream(dh)),
           "moe_swiglu_backward")
    return du


def moe_expert_backward(dy: torch.Tensor, p: "Permuted", routing_w: torch.Tensor, w_ug: torch.Tensor,
                        w_down: torch.Tensor, h_buf: torch.Tensor, y_perm: torch.Tensor, u: torch.Tensor | None = None
                        ) -> dict:
    """The expert step's backward from its forward tensors (``p`` must hold x_perm): returns dx,
    d_routing_w, dw_ug, dw_down. ``u`` is the pre-activation kept by moe_gemm_up_swiglu_u; without it, U is
    recomputed with the gate/up projection. Every step is one of the library's calls above."""
    if p.x_perm is None:
        raise ValueError("the backward needs the permuted rows: run moe_permute with gather=True")
    dy_perm, d_rw = moe_unpermute_backward(dy, y_perm, p.inv_map, routing_w)
    dh = moe_grouped_dgrad(dy_perm, p.offsets, w_down, "in_out")
    dw_down = moe_grouped_wgrad(h_buf, dy_perm, p.offsets, "in_out")
    if u is None:
        u = moe_grouped_projection(p.x_perm, p.offsets, w_ug, "out_in")
    du = moe_swiglu_backward(dh, u, p.offsets)
    dx_perm = moe_grouped_dgrad(du, p.offsets, w_ug, "out_in")
    dw_ug = moe_grouped_wgrad(p.x_perm, du, p.offsets, "out_in")
    dx = moe_permute_backward(dx_perm, p.inv_map)
    return {"dx": dx, "d_routing_w": d_rw, "dw_ug": dw_ug, "dw_down": dw_down, "dy_perm": dy_perm, "dh": dh,
            "u": u, "du": du, "dx_perm": dx_perm}


def moe_grouped_dgrad(dy: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor, layout: str = "in_out", *,
                      dx=None) -> torch.Tensor:
    """dX[rows_e] = bf16(dY[rows_e] @ W_e^T) for the projection Y_e = X_e W_e (one launch)."""
    E, d_in, d_out = _w_dims(w, layout)
    if dy.dim() != 2:
        raise ValueError("dy must be [cap_rows, d_out]")
    cap, dev = dy.shape[0], dy.device
    _want(dy, "dy", torch.bfloat16, (cap, d_out), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    _want(w, "w", torch.bfloat16, tuple(w.shape), dev)
    dx = _out(dx, "dx", torch.bfloat16, (cap, d_in), dev)
    _check(load_library().moe_grouped_dgrad(_ptr(dy), _ptr(offsets), _ptr(w), W_LAYOUTS[layout], cap, d_in, d_out, E,
                                            _ptr(dx), _stream(dy)), "moe_grouped_dgrad")
    return dx


def wgrad_workspace_bytes(cap_rows: int, d_in: int, d_out: int, E: int) -> int:
    return int(load_library().moe_grouped_wgrad_workspace_bytes(cap_rows, d_in, d_out, E))


def moe_grouped_wgrad(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, layout: str = "in_out", *,
                      dw=None, workspace=None) -> torch.Tensor:
    """dW_e = bf16(X[rows_e]^T @ dY[rows_e]) in the weight's layout; zeros for experts with no rows (one launch)."""
    if x.dim() != 2 or dy.dim() != 2 or offsets.dim() != 1:
        raise ValueError("expected x [cap, d_in], dy [cap, d_out] and offsets [E+1]")
    cap, d_in = x.shape
    d_out = dy.shape[1]
    E = offsets.shape[0] - 1
    dev = x.device
    _want(x, "x", torch.bfloat16, (cap, d_in), dev)
    _want(dy, "dy", torch.bfloat16, (cap, d_out), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    if layout not in W_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(W_LAYOUTS)}, got {layout!r}")
    shape = (E, d_in, d_out) if layout == "in_out" else (E, d_out, d_in)
    dw = _out(dw, "dw", torch.bfloat16, shape, dev)
    need = wgrad_workspace_bytes(cap, d_in, d_out, E)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    if (workspace.device != dev or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {dev}")
    _check(load_library().moe_grouped_wgrad(_ptr(x), _ptr(dy), _ptr(offsets), W_LAYOUTS[layout], cap, d_in, d_out, E,
                                            _ptr(dw), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(x)), "moe_grouped_wgrad")
    return dw


def moe_permute_backward(dx_perm: torch.Tensor, inv_map: torch.Tensor, *, dx=None) -> torch.Tensor:
    """dX[t] = bf16(sum over kept j of dx_perm[inv_map[t, j]]) (gather + reduce, no atomics)."""
    if inv_map.dim() != 2:
        raise ValueError("inv_map must be [T, k]")
    T, k = inv_map.shape
    dev = dx_perm.device
    d = dx_perm.shape[1]
    _want(dx_perm, "dx_perm", torch.bfloat16, (T * k, d), dev)
    _want(inv_map, "inv_map", torch.int32, (T, k), dev)
    dx = _out(dx, "dx", torch.bfloat16, (T, d), dev)
    _check(load_library().moe_permute_backward(_ptr(dx_perm), _ptr(inv_map), T, k, d, _ptr(dx), _stream(dx_perm)),
           "moe_permute_backward")
    return dx


def moe_unpermute_backward(dy: torch.Tensor, y_perm: torch.Tensor, inv_map: torch.Tensor, routing_w: torch.Tensor, *,
                           dy_perm=None, d_routing_w=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Backward of moe_unpermute: (dy_perm with rows inv_map[t, j] = bf16(w[t, j] * dy[t]), d_routing_w fp32)."""
    if inv_map.dim() != 2:
        raise ValueError("inv_map must be [T, k]")
    T, k = inv_map.shape
    dev = dy.device
    d = dy.shape[1]
    _want(dy, "dy", torch.bfloat16, (T, d), dev)
    _want(y_perm, "y_perm", torch.bfloat16, (T * k, d), dev)
    _want(inv_map, "inv_map", torch.int32, (T, k), dev)
    _want(routing_w, "routing_w", torch.float32, (T, k), dev)
    dy_perm = _out(dy_perm, "dy_perm", torch.bfloat16, (T * k, d), dev)
    d_routing_w = _out(d_routing_w, "d_routing_w", torch.float32, (T, k), dev)
    _check(load_library().moe_unpermute_backward(_ptr(dy), _ptr(y_perm), _ptr(inv_map), _ptr(routing_w), T, k, d,
                                                 _ptr(dy_perm), _ptr(d_routing_w), _stream(dy)),
           "moe_unpermute_backward")
    return dy_perm, d_routing_w


def moe_expert_forward(x, expert_ids, routing_w, w_ug, w_down, fused_gather: bool = False):
    """The whole step: permute, grouped SwiGLU expert, unpermute. Returns (y, Permuted, h_buf, y_perm).

    ``fused_gather=True`` skips x_perm: the gate/up GEMM reads X through perm.
    """
    p = moe_permute(x, expert_ids, w_ug.shape[0], gather=not fused_gather)
    if fused_gather:
        h_buf, y_perm = grouped_swiglu_expert_gather(x, p.perm, p.offsets, w_ug, w_down, expert_ids.shape[1])
    else:
        h_buf, y_perm = grouped_swiglu_expert(p.x_perm, p.offsets, w_ug, w_down)
    y = moe_unpermute(y_perm, p.inv_map, routing_w)
    return y, p, h_buf, y_perm


# ------------------------------------------------------------------ router

_LOGITS = {torch.bfloat16: 0, torch.float32: 1}
ROUTER_MAX_TOPK = 64


@dataclass
class Routed:
    expert_ids: torch.Tensor  # int32 [T, k]; -1 for a slot left over by the mask
    routing_w: torch.Tensor  # fp32 [T, k]
    lse: torch.Tensor  # fp32 [T]
    renormalize: bool
    counts: torch.Tensor | None = None  # int32 [E]; these four from moe_router_topk_losses only
    tokens: torch.Tensor | None = None  # int32 [1]
    prob_mean: torch.Tensor | None = None  # fp32 [E]
    losses: torch.Tensor | None = None  # fp32 [2]: balance loss, z-loss


def _logits(logits: torch.Tensor, k: int):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    dtype, dev, (T, E) = logits.dtype, logits.device, logits.shape
    code = _LOGITS.get(dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16 or float32, got {dtype}")
    _want(logits, "logits", dtype, (T, E), dev)
    if not (1 <= k <= E and k <= ROUTER_MAX_TOPK):
        raise ValueError(f"k must be between 1 and min(E, {ROUTER_MAX_TOPK}), got {k} for E = {E}")
    return T, E, code, dev


def moe_router_topk(logits: torch.Tensor, k: int, *, renormalize: bool = True, expert_ids=None, routing_w=None,
                    lse=None) -> Routed:
    """The k largest logits of every row (lowest index first among equals), their softmax weights and the row's
    log-sum-exp (one launch). Experts at -inf are never chosen: their slots get id -1 and weight 0."""
    T, E, dtype, dev = _logits(logits, k)
    expert_ids = _out(expert_ids, "expert_ids", torch.int32, (T, k), dev)
    routing_w = _out(routing_w, "routing_w", torch.float32, (T, k), dev)
    lse = _out(lse, "lse", torch.float32, (T,), dev)
    _check(load_library().moe_router_topk(logits.data_ptr(), dtype, T, E, k, int(renormalize), expert_ids.data_ptr(),
                                          routing_w.data_ptr(), lse.data_ptr(), _stream(logits)), "moe_router_topk")
    return Routed(expert_ids, routing_w, lse, bool(renormalize))


def router_workspace_bytes(T: int, E: int) -> int:
    return int(load_library().moe_router_workspace_bytes(T, E))


def moe_router_topk_losses(logits: torch.Tensor, k: int, *, renormalize: bool = True, expert_ids=None, routing_w=None,
                           lse=None, counts=None, tokens=None, prob_mean=None, losses=None, workspace=None) -> Routed:
    """moe_router_topk with the per-expert counts, the mean probabilities, and losses = [balance, z] (two launches)."""
    T, E, dtype, dev = _logits(logits, k)
    expert_ids = _out(expert_ids, "expert_ids", torch.int32, (T, k), dev)
    routing_w = _out(routing_w, "routing_w", torch.float32, (T, k), dev)
    lse = _out(lse, "lse", torch.float32, (T,), dev)
    if counts is None and tokens is None and prob_mean is None and losses is None:
        # one allocation for the four
        words = torch.empty((2 * E + 3,), dtype=torch.int32, device=dev)
        counts, tokens, prob_mean, losses = words.split_with_sizes((E, 1, E, 2))
        prob_mean, losses = prob_mean.view(torch.float32), losses.view(torch.float32)
    else:
        counts = _out(counts, "counts", torch.int32, (E,), dev)
        tokens = _out(tokens, "tokens", torch.int32, (1,), dev)
        prob_mean = _out(prob_mean, "prob_mean", torch.float32, (E,), dev)
        losses = _out(losses, "losses", torch.float32, (2,), dev)
    if workspace is None:
        workspace = torch.empty((router_workspace_bytes(T, E),), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    _check(load_library().moe_router_topk_losses(logits.data_ptr(), dtype, T, E, k, int(renormalize),
                                                 expert_ids.data_ptr(), routing_w.data_ptr(), lse.data_ptr(),
                                                 counts.data_ptr(), tokens.data_ptr(), prob_mean.data_ptr(),
                                                 losses.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                                 _stream(logits)), "moe_router_topk_losses")
    return Routed(expert_ids, routing_w, lse, bool(renormalize), counts, tokens, prob_mean, losses)


def moe_router_backward(logits: torch.Tensor, routed: Routed, d_routing_w: torch.Tensor | None = None,
                        d_losses: torch.Tensor | None = None, *, d_logits=None) -> torch.Tensor:
    """Gradient of the logits from those of the routing weights ([T, k] fp32) and of the losses ([2] fp32, on the
    device); either may be None (one launch). For losses over several ranks' tokens, sum ``routed.counts`` and
    ``routed.tokens`` over the ranks first."""
    k = routed.expert_ids.shape[1]
    T, E, dtype, dev = _logits(logits, k)
    _want(routed.expert_ids, "expert_ids", torch.int32, (T, k), dev)
    _want(routed.routing_w, "routing_w", torch.float32, (T, k), dev)
    if d_routing_w is not None:
        _want(d_routing_w, "d_routing_w", torch.float32, (T, k), dev)
    if d_losses is not None:
        if routed.counts is None or routed.tokens is None:
            raise ValueError("the gradient of the losses needs the counts of moe_router_topk_losses")
        _want(d_losses, "d_losses", torch.float32, (2,), dev)
        _want(routed.counts, "counts", torch.int32, (E,), dev)
        _want(routed.tokens, "tokens", torch.int32, (1,), dev)
    d_logits = _out(d_logits, "d_logits", logits.dtype, (T, E), dev)
    _check(load_library().moe_router_backward(logits.data_ptr(), dtype, T, E, k, int(routed.renormalize),
                                              routed.expert_ids.data_ptr(), routed.routing_w.data_ptr(), _ptr(routed.counts),
                                              _ptr(routed.tokens), _ptr(d_routing_w), _ptr(d_losses), d_logits.data_ptr(),
                                              _stream(logits)), "moe_router_backward")
    return d_logits


# ------------------------------------------------------------------ MXFP4


@dataclass
class Mxfp4:
    """Rows of ``width`` 4-bit values with a power of two per 32: q [..., 16 * ceil(width / 32)] and
    scales [..., 16 * ceil(width / 512)], both uint8."""
    q: torch.Tensor
    scales: torch.Tensor
    width: int


def mxfp4_row_bytes(width: int) -> int:
    return 16 * ((width + 31) // 32)


def mxfp4_scale_bytes(width: int) -> int:
    return 16 * ((width + 511) // 512)


def _want_mxfp4(m: Mxfp4, name: str, lead: tuple, device) -> None:
    if not isinstance(m, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4")
    _want(m.q, f"{name}.q", torch.uint8, (*lead, mxfp4_row_bytes(m.width)), device)
    _want(m.scales, f"{name}.scales", torch.uint8, (*lead, mxfp4_scale_bytes(m.width)), device)


def moe_mxfp4_quantize(x: torch.Tensor, *, q=None, scales=None) -> Mxfp4:
    """bf16 rows [..., K] to MXFP4 along the last dimension (one launch)."""
    if x.dim() < 1:
        raise ValueError("x must have a last dimension to quantise along")
    _want(x, "x", torch.bfloat16, tuple(x.shape), x.device)
    lead, K = tuple(x.shape[:-1]), x.shape[-1]
    q = _out(q, "q", torch.uint8, (*lead, mxfp4_row_bytes(K)), x.device)
    scales = _out(scales, "scales", torch.uint8, (*lead, mxfp4_scale_bytes(K)), x.device)
    rows = 1
    for n in lead:
        rows *= n
    _check(load_library().moe_mxfp4_quantize(x.data_ptr(), rows, K, q.data_ptr(), scales.data_ptr(), _stream(x)),
           "moe_mxfp4_quantize")
    return Mxfp4(q, scales, K)


def moe_mxfp4_quantize_weights(w: torch.Tensor, layout: str = "in_out", *, q=None, scales=None) -> Mxfp4:
    """Expert weights [E, d_in, d_out] ("in_out") or [E, d_out, d_in] ("out_in") to MXFP4 rows [E, d_out] of d_in
    values, the form the MXFP4 products read (one launch)."""
    E, d_in, d_out = _w_dims(w, layout)
    dev = w.device
    _want(w, "w", torch.bfloat16, tuple(w.shape), dev)
    q = _out(q, "q", torch.uint8, (E, d_out, mxfp4_row_bytes(d_in)), dev)
    scales = _out(scales, "scales", torch.uint8, (E, d_out, mxfp4_scale_bytes(d_in)), dev)
    _check(load_library().moe_mxfp4_quantize_weights(w.data_ptr(), W_LAYOUTS[layout], d_in, d_out, E, q.data_ptr(),
                                                     scales.data_ptr(), _stream(w)), "moe_mxfp4_quantize_weights")
    return Mxfp4(q, scales, d_in)


def moe_mxfp4_dequantize(m: Mxfp4, *, x=None) -> torch.Tensor:
    """The bf16 values of MXFP4 rows (one launch). Exact for scale bytes up to 252, which the quantising calls do not
    pass; at 253 and 254 a value past bf16's range is an infinity."""
    if not isinstance(m, Mxfp4) or m.q.dim() < 1:
        raise TypeError("expected an Mxfp4")
    lead, dev = tuple(m.q.shape[:-1]), m.q.device
    _want_mxfp4(m, "m", lead, dev)
    x = _out(x, "x", torch.bfloat16, (*lead, m.width), dev)
    rows = 1
    for n in lead:
        rows *= n
    _check(load_library().moe_mxfp4_dequantize(m.q.data_ptr(), m.scales.data_ptr(), rows, m.width, x.data_ptr(),
                                               _stream(m.q)), "moe_mxfp4_dequantize")
    return x


def _mxfp4_experts(x: Mxfp4, offsets: torch.Tensor, w: Mxfp4):
    if not isinstance(x, Mxfp4) or not isinstance(w, Mxfp4) or x.q.dim() != 2 or w.q.dim() != 3:
        raise ValueError("expected Mxfp4 rows [rows, .] and Mxfp4 expert weights [E, d_out, .]")
    if x.width != w.width:
        raise ValueError(f"rows of {x.width} values do not fit weights of {w.width}")
    q, dev = mxfp4_row_bytes(x.width), x.q.device
    s = mxfp4_scale_bytes(x.width)
    rows, (E, w_rows, _) = x.q.shape[0], w.q.shape
    _want(x.q, "x.q", torch.uint8, (rows, q), dev)
    _want(x.scales, "x.scales", torch.uint8, (rows, s), dev)
    _want(w.q, "w.q", torch.uint8, (E, w_rows, q), dev)
    _want(w.scales, "w.scales", torch.uint8, (E, w_rows, s), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    return rows, E, w_rows, dev


def moe_grouped_projection_mxfp4(x: Mxfp4, offsets: torch.Tensor, w: Mxfp4, *, y=None) -> torch.Tensor:
    """Y[rows_e] = bf16(X[rows_e] @ W_e^T) on MXFP4 rows [cap, d_in] and weights [E, d_out, d_in] (one launch)."""
    cap, E, d_out, dev = _mxfp4_experts(x, offsets, w)
    y = _out(y, "y", torch.bfloat16, (cap, d_out), dev)
    _check(load_library().moe_grouped_projection_mxfp4(x.q.data_ptr(), x.scales.data_ptr(), offsets.data_ptr(),
                                                       w.q.data_ptr(), w.scales.data_ptr(), cap, x.width, d_out, E,
                                                       y.data_ptr(), _stream(x.q)), "moe_grouped_projection_mxfp4")
    return y


def _mxfp4_up(x: Mxfp4, offsets: torch.Tensor, w_ug: Mxfp4, perm, k: int):
    T, E, two_h, dev = _mxfp4_experts(x, offsets, w_ug)
    if two_h % 2:
        raise ValueError("w_ug must hold as many gate as up rows")
    k = int(k)
    if perm is not None:
        _want(perm, "perm", torch.int32, (T * k,), dev)
    elif k != 1:
        raise ValueError("k other than 1 needs perm")
    return T, k, E, two_h // 2, dev


def moe_gemm_up_swiglu_mxfp4(x: Mxfp4, offsets: torch.Tensor, w_ug: Mxfp4, *, perm=None, k: int = 1,
                             h_buf=None) -> torch.Tensor:
    """h_buf[p] = bf16(SiLU(g) * u), [g | u] = X[perm[p] // k] @ W_ug[e]^T, on MXFP4 token rows [T, d] and weights
    [E, 2h, d] (one launch). Without ``perm`` the rows are sorted already and k is 1."""
    T, k, E, h, dev = _mxfp4_up(x, offsets, w_ug, perm, k)
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (T * k, h), dev)
    _check(load_library().moe_gemm_up_swiglu_mxfp4(x.q.data_ptr(), x.scales.data_ptr(), _ptr(perm), T, k,
                                                   offsets.data_ptr(), w_ug.q.data_ptr(), w_ug.scales.data_ptr(),
                                                   x.width, h, E, h_buf.data_ptr(), _stream(x.q)),
           "moe_gemm_up_swiglu_mxfp4")
    return h_buf


def moe_gemm_up_swiglu_mxfp4_q(x: Mxfp4, offsets: torch.Tensor, w_ug: Mxfp4, *, perm=None, k: int = 1, q=None,
                               scales=None) -> Mxfp4:
    """moe_gemm_up_swiglu_mxfp4 with its result quantised in the same launch, bit for bit as moe_mxfp4_quantize
    would: MXFP4 rows [T * k] of h values for the down projection."""
    T, k, E, h, dev = _mxfp4_up(x, offsets, w_ug, perm, k)
    q = _out(q, "q", torch.uint8, (T * k, mxfp4_row_bytes(h)), dev)
    scales = _out(scales, "scales", torch.uint8, (T * k, mxfp4_scale_bytes(h)), dev)
    _check(load_library().moe_gemm_up_swiglu_mxfp4_q(x.q.data_ptr(), x.scales.data_ptr(), _ptr(perm), T, k,
                                                     offsets.data_ptr(), w_ug.q.data_ptr(), w_ug.scales.data_ptr(),
                                                     x.width, h, E, q.data_ptr(), scales.data_ptr(), _stream(x.q)),
           "moe_gemm_up_swiglu_mxfp4_q")
    return Mxfp4(q, scales, h)


def moe_expert_forward_mxfp4(x: torch.Tensor, expert_ids: torch.Tensor, routing_w: torch.Tensor, w_ug: Mxfp4,
                             w_down: Mxfp4):
    """The whole step on MXFP4 experts, from bf16 token rows: the rows and the SwiGLU activations are quantised on the
    way. ``w_ug`` holds [E, 2h] rows of d values, ``w_down`` [E, d] rows of h (moe_mxfp4_quantize_weights of the bf16
    weights). Returns (y, Permuted)."""
    k = expert_ids.shape[1]
    p = moe_permute(x, expert_ids, w_ug.q.shape[0], gather=False)
    h = moe_gemm_up_swiglu_mxfp4_q(moe_mxfp4_quantize(x), p.offsets, w_ug, perm=p.perm, k=k)
    y_perm = moe_grouped_projection_mxfp4(h, p.offsets, w_down)
    return moe_unpermute(y_perm, p.inv_map, routing_w), p


# ------------------------------------------------------------------ 4-bit weights with group scales


@dataclass
class Int4:
    """Expert weights [E, d_out, width] as s (q - z): q uint8 [E, d_out, 16 * ceil(width / 32)], scales bf16 and zeros
    uint8 (None: 8 everywhere) [E, ceil(width / group), d_out]."""
    q: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None
    width: int
    group: int = 128


INT4_GROUPS = (32, 64, 128)


def _int4_shapes(E: int, d_out: int, width: int, group: int):
    if group not in INT4_GROUPS:
        raise ValueError(f"group must be one of {INT4_GROUPS}, got {group}")
    return (E, d_out, 16 * ((width + 31) // 32)), (E, (width + group - 1) // group, d_out)


def _want_int4(w: Int4, name: str, device):
    if not isinstance(w, Int4):
        raise TypeError(f"{name} must be an Int4")
    if not isinstance(w.q, torch.Tensor) or w.q.dim() != 3:
        raise ValueError(f"{name}.q must be [E, d_out, .]")
    E, d_out, _ = w.q.shape
    q, s = _int4_shapes(E, d_out, w.width, w.group)
    _want(w.q, f"{name}.q", torch.uint8, q, device)
    _want(w.scales, f"{name}.scales", torch.bfloat16, s, device)
    if w.zeros is not None:
        _want(w.zeros, f"{name}.zeros", torch.uint8, s, device)
    return E, d_out


def moe_int4_quantize_weights(w: torch.Tensor, layout: str = "in_out", *, group: int = 128, symmetric: bool = False,
                              q=None, scales=None, zeros=None) -> Int4:
    """Expert weights [E, d_in, d_out] ("in_out") or [E, d_out, d_in] ("out_in") rounded to 4 bits with a scale, and
    unless ``symmetric`` a zero, for every ``group`` values of the contraction (one launch)."""
    E, d_in, d_out = _w_dims(w, layout)
    dev = w.device
    _want(w, "w", torch.bfloat16, tuple(w.shape), dev)
    q_shape, s_shape = _int4_shapes(E, d_out, d_in, group)
    q = _out(q, "q", torch.uint8, q_shape, dev)
    scales = _out(scales, "scales", torch.bfloat16, s_shape, dev)
    if symmetric and zeros is not None:
        raise ValueError("symmetric weights have no zeros")
    zeros = None if symmetric else _out(zeros, "zeros", torch.uint8, s_shape, dev)
    _check(load_library().moe_int4_quantize_weights(w.data_ptr(), W_LAYOUTS[layout], d_in, d_out, E, group, q.data_ptr(),
                                                    scales.data_ptr(), _ptr(zeros), _stream(w)),
           "moe_int4_quantize_weights")
    return Int4(q, scales, zeros, d_in, group)


def moe_int4_dequantize_weights(m: Int4, *, w=None) -> torch.Tensor:
    """The bf16 weights [E, d_out, d_in] ("out_in") of packed ones, for the bf16 calls (one launch)."""
    if not isinstance(m, Int4):
        raise TypeError("expected an Int4")
    dev = m.q.device
    E, d_out = _want_int4(m, "m", dev)
    w = _out(w, "w", torch.bfloat16, (E, d_out, m.width), dev)
    _check(load_library().moe_int4_dequantize_weights(m.q.data_ptr(), m.scales.data_ptr(), _ptr(m.zeros), m.width, d_out,
                                                      E, m.group, w.data_ptr(), _stream(m.q)),
           "moe_int4_dequantize_weights")
    return w


def moe_grouped_projection_int4(x: torch.Tensor, offsets: torch.Tensor, w: Int4, *, y=None) -> torch.Tensor:
    """Y[rows_e] = bf16(X[rows_e] @ W_e^T) of bf16 rows [cap, d_in] and 4-bit weights [E, d_out, d_in] (one launch).
    From about 200 rows an expert on, moe_int4_dequantize_weights and moe_grouped_projection are faster."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [cap_rows, d_in]")
    dev = x.device
    E, d_out = _want_int4(w, "w", dev)
    cap = x.shape[0]
    _want(x, "x", torch.bfloat16, (cap, w.width), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    y = _out(y, "y", torch.bfloat16, (cap, d_out), dev)
    _check(load_library().moe_grouped_projection_int4(x.data_ptr(), offsets.data_ptr(), w.q.data_ptr(),
                                                      w.scales.data_ptr(), _ptr(w.zeros), w.group, cap, w.width, d_out,
                                                      E, y.data_ptr(), _stream(x)), "moe_grouped_projection_int4")
    return y


def moe_gemm_up_swiglu_int4(x: torch.Tensor, offsets: torch.Tensor, w_ug: Int4, *, perm=None, k: int = 1,
                            h_buf=None) -> torch.Tensor:
    """h_buf[p] = bf16(SiLU(g) * u), [g | u] = X[perm[p] // k] @ W_ug[e]^T, of bf16 token rows [T, d] and 4-bit weights
    [E, 2h, d] (one launch). Without ``perm`` the rows are sorted already and k is 1."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [T, d]")
    dev = x.device
    E, two_h = _want_int4(w_ug, "w_ug", dev)
    T, k = x.shape[0], int(k)
    _want(x, "x", torch.bfloat16, (T, w_ug.width), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    if two_h % 2:
        raise ValueError("w_ug must hold as many gate as up rows")
    if perm is not None:
        _want(perm, "perm", torch.int32, (T * k,), dev)
    elif k != 1:
        raise ValueError("k other than 1 needs perm")
    h_buf = _out(h_buf, "h_buf", torch.bfloat16, (T * k, two_h // 2), dev)
    _check(load_library().moe_gemm_up_swiglu_int4(x.data_ptr(), _ptr(perm), T, k, offsets.data_ptr(), w_ug.q.data_ptr(),
                                                  w_ug.scales.data_ptr(), _ptr(w_ug.zeros), w_ug.group, w_ug.width,
                                                  two_h // 2, E, h_buf.data_ptr(), _stream(x)),
           "moe_gemm_up_swiglu_int4")
    return h_buf


def moe_expert_forward_int4(x: torch.Tensor, expert_ids: torch.Tensor, routing_w: torch.Tensor, w_ug: Int4,
                            w_down: Int4):
    """The whole step on 4-bit experts, from bf16 token rows. ``w_ug`` holds [E, 2h] rows of d values, ``w_down``
    [E, d] rows of h (moe_int4_quantize_weights of the bf16 weights). Returns (y, Permuted). For decode and small batches:
    from about 200 rows an expert on, moe_expert_forward on weights read back with moe_int4_dequantize_weights is faster."""
    k = expert_ids.shape[1]
    p = moe_permute(x, expert_ids, w_ug.q.shape[0], gather=False)
    h = moe_gemm_up_swiglu_int4(x, p.offsets, w_ug, perm=p.perm, k=k)
    y_perm = moe_grouped_projection_int4(h, p.offsets, w_down)
    return moe_unpermute(y_perm, p.inv_map, routing_w), p


# ------------------------------------------------------------------ norms around a block

NORM_MAX_WIDTH = 16384
_NORM_POST, _NORM_NEXT = 1, 2
_GATE_NONE, _GATE_TOKEN, _GATE_CHANNEL = 0, 1, 2


def _stream_rows(r: torch.Tensor, name: str):
    """(T, d, dtype code, device) of rows of the residual stream."""
    if not isinstance(r, torch.Tensor) or r.dim() != 2:
        raise ValueError(f"{name} must be [T, d]")
    code = _LOGITS.get(r.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {r.dtype}")
    T, d = r.shape
    dev = r.device
    _want(r, name, r.dtype, (T, d), dev)
    return T, d, code, dev


def _norm_weights(shape: tuple, dev, *weights) -> int:
    """dtype code of the (weight, name) pairs whose weight is given, all of one dtype."""
    dtype = code = None
    for w, name in weights:
        if w is None:
            continue
        if code is None:
            dtype = w.dtype if isinstance(w, _Tensor) else None
            code = _LOGITS.get(dtype)
            if code is None:
                raise TypeError(f"{name} must be a bfloat16 or float32 tensor")
        _want(w, name, dtype, shape, dev)
    return code or 0


def _norm_gate(gate, T: int, d: int, dev):
    """(kind, the gate if it is one per channel)"""
    if gate is None:
        return _GATE_NONE, None
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        _want(gate, "gate", torch.float32, (T, 1), dev)
        return _GATE_TOKEN, None
    return _GATE_CHANNEL, gate


@functools.lru_cache(maxsize=256)
def norm_workspace_bytes(T: int, d: int) -> int:
    return int(load_library().moe_norm_workspace_bytes(T, d))


def _norm_workspace(workspace, T: int, d: int, dev):
    if workspace is None:
        return torch.empty((norm_workspace_bytes(T, d),), dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    return workspace


def moe_rmsnorm(x: torch.Tensor, w: torch.Tensor | None = None, *, eps: float = 1e-6, y=None) -> torch.Tensor:
    """The norm before a block: bf16 rows x / sqrt(mean(x^2) + eps) * w of the stream's bf16 or fp32 rows (one launch)."""
    T, d, dtype, dev = _stream_rows(x, "x")
    w_dtype = _norm_weights((d,), dev, (w, "w"))
    y = _out(y, "y", torch.bfloat16, (T, d), dev)
    _check(load_library().moe_rmsnorm(x.data_ptr(), dtype, _ptr(w), w_dtype, eps, T, d, y.data_ptr(), _stream(x)),
           "moe_rmsnorm")
    return y


def moe_rmsnorm_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor | None = None, *, eps: float = 1e-6,
                         dy_add=None, dx_add=None, dx=None, dw=None, workspace=None):
    """(dx, dw) of moe_rmsnorm: dx in the stream's type with ``dx_add``, the gradient that reaches x past the norm,
    added; dw fp32, None without a weight (two launches). ``dy_add`` is a second part of y's gradient."""
    T, d, dtype, dev = _stream_rows(x, "x")
    w_dtype = _norm_weights((d,), dev, (w, "w"))
    _want(dy, "dy", torch.bfloat16, (T, d), dev)
    if dy_add is not None:
        _want(dy_add, "dy_add", torch.bfloat16, (T, d), dev)
    if dx_add is not None:
        _want(dx_add, "dx_add", x.dtype, (T, d), dev)
    dx = _out(dx, "dx", x.dtype, (T, d), dev)
    dw = None if w is None else _out(dw, "dw", torch.float32, (d,), dev)
    workspace = _norm_workspace(workspace, T, d, dev)
    _check(load_library().moe_rmsnorm_backward(dy.data_ptr(), _ptr(dy_add), x.data_ptr(), dtype, _ptr(w), w_dtype, eps,
                                               _ptr(dx_add), T, d, dx.data_ptr(), _ptr(dw), workspace.data_ptr(), workspace.numel(),
                                               _stream(x)), "moe_rmsnorm_backward")
    return dx, dw


def moe_residual_norm(y: torch.Tensor, r: torch.Tensor, *, post_norm: bool = False, w_post=None, gate=None,
                      residual_scale: float = 1.0, branch_scale: float = 1.0, next_norm: bool = True, w_next=None,
                      eps: float = 1e-6, r_out=None, n_out=None):
    """What follows a block: r' = residual_scale * r + branch_scale * gate * u with u = RMSNorm(y) * w_post
    (``post_norm``) or y, and n = RMSNorm(r') * w_next for the block behind (``next_norm``). ``gate`` is fp32 [T, 1],
    a number a token, or [d], a number a channel. Returns (r', n), n None without the next norm (one launch)."""
    T, d, dtype, dev = _stream_rows(r, "r")
    _want(y, "y", torch.bfloat16, (T, d), dev)
    kind, channel = _norm_gate(gate, T, d, dev)
    if (w_post is not None and not post_norm) or (w_next is not None and not next_norm):
        raise ValueError("a weight of a norm that is not asked for")
    w_dtype = _norm_weights((d,), dev, (w_post, "w_post"), (w_next, "w_next"), (channel, "gate"))
    r_out = _out(r_out, "r_out", r.dtype, (T, d), dev)
    n_out = _out(n_out, "n_out", torch.bfloat16, (T, d), dev) if next_norm else None
    flags = (_NORM_POST if post_norm else 0) | (_NORM_NEXT if next_norm else 0)
    _check(load_library().moe_residual_norm(y.data_ptr(), r.data_ptr(), dtype, flags, _ptr(w_post), _ptr(w_next), w_dtype,
                                            _ptr(gate), kind, residual_scale, branch_scale, eps, T, d, r_out.data_ptr(),
                                            _ptr(n_out), _stream(r)), "moe_residual_norm")
    return r_out, n_out


@dataclass
class ResidualNormGrads:
    d_r: torch.Tensor  # the stream's type [T, d]
    d_y: torch.Tensor  # bf16 [T, d]
    d_gate: torch.Tensor | None  # fp32, the gate's shape
    d_w_post: torch.Tensor | None  # fp32 [d]
    d_w_next: torch.Tensor | None  # fp32 [d]


def moe_residual_norm_backward(d_r_out: torch.Tensor | None, d_n: torch.Tensor | None, y: torch.Tensor,
                               r_out: torch.Tensor, *, post_norm: bool = False, w_post=None, gate=None,
                               residual_scale: float = 1.0, branch_scale: float = 1.0, next_norm: bool = True,
                               w_next=None, eps: float = 1e-6, d_n_add=None, d_r=None, d_y=None, d_gate=None,
                               d_w_post=None, d_w_next=None, workspace=None) -> ResidualNormGrads:
    """Gradients of moe_residual_norm from those of r' (None: none) and n (``d_n_add``: a second part of it), with the
    block's output y and r' as the forward wrote it; weights' and gate's in fp32 (two launches)."""
    T, d, dtype, dev = _stream_rows(r_out, "r_out")
    _want(y, "y", torch.bfloat16, (T, d), dev)
    kind, channel = _norm_gate(gate, T, d, dev)
    if (w_post is not None and not post_norm) or (w_next is not None and not next_norm):
        raise ValueError("a weight of a norm that is not asked for")
    w_dtype = _norm_weights((d,), dev, (w_post, "w_post"), (w_next, "w_next"), (channel, "gate"))
    if d_r_out is not None:
        _want(d_r_out, "d_r_out", r_out.dtype, (T, d), dev)
    elif not next_norm:
        raise ValueError("without the next norm the only gradient is that of r_out")
    if next_norm:
        _want(d_n, "d_n", torch.bfloat16, (T, d), dev)
        if d_n_add is not None:
            _want(d_n_add, "d_n_add", torch.bfloat16, (T, d), dev)
    elif d_n is not None or d_n_add is not None:
        raise ValueError("a gradient of a norm that is not asked for")
    d_r = _out(d_r, "d_r", r_out.dtype, (T, d), dev)
    d_y = _out(d_y, "d_y", torch.bfloat16, (T, d), dev)
    d_gate = None if gate is None else _out(d_gate, "d_gate", torch.float32, tuple(gate.shape), dev)
    d_w_post = None if w_post is None else _out(d_w_post, "d_w_post", torch.float32, (d,), dev)
    d_w_next = None if w_next is None else _out(d_w_next, "d_w_next", torch.float32, (d,), dev)
    workspace = _norm_workspace(workspace, T, d, dev)
    flags = (_NORM_POST if post_norm else 0) | (_NORM_NEXT if next_norm else 0)
    _check(load_library().moe_residual_norm_backward(
        _ptr(d_r_out), _ptr(d_n), _ptr(d_n_add), y.data_ptr(), r_out.data_ptr(), dtype, flags, _ptr(w_post),
        _ptr(w_next), w_dtype, _ptr(gate), kind, residual_scale, branch_scale, eps, T, d, d_r.data_ptr(), d_y.data_ptr(),
        _ptr(d_gate), _ptr(d_w_post), _ptr(d_w_next), workspace.data_ptr(), workspace.numel(), _stream(r_out)),
        "moe_residual_norm_backward")
    return ResidualNormGrads(d_r, d_y, d_gate, d_w_post, d_w_next)


# ------------------------------------------------------------------ a layer on the residual stream


@dataclass
class MoeLayer:
    """What moe_layer_forward gives: the stream behind the layer, the next norm's rows if asked for, and what the backward
    reads."""
    r_out: torch.Tensor
    n_out: torch.Tensor | None
    routed: Routed
    p: Permuted
    r: torch.Tensor
    n: torch.Tensor  # the rows the router and the experts read
    logits: torch.Tensor
    rows: torch.Tensor  # int32 [2]: the router's product has one group
    h_buf: torch.Tensor
    u: torch.Tensor
    y_perm: torch.Tensor
    y: torch.Tensor
    eps: float
    after: dict  # arguments of moe_residual_norm


def moe_layer_forward(r: torch.Tensor, w_norm, w_router: torch.Tensor, w_ug: torch.Tensor, w_down: torch.Tensor, k: int,
                      *, renormalize: bool = True, eps: float = 1e-6, post_norm: bool = False, w_post=None, gate=None,
                      residual_scale: float = 1.0, branch_scale: float = 1.0, next_norm: bool = False,
                      w_next=None) -> MoeLayer:
    """A routed layer on the residual stream ``r``, bf16 or fp32 [T, d]: norm, router (``w_router`` bf16 [E, d], E a
    multiple of 8), experts, and moe_residual_norm with the arguments after ``eps``. Its losses are in ``routed``."""
    n = moe_rmsnorm(r, w_norm, eps=eps)
    rows = torch.arange(2, dtype=torch.int32, device=r.device) * r.shape[0]
    logits = moe_grouped_projection(n, rows, w_router[None], "out_in")
    routed = moe_router_topk_losses(logits, k, renormalize=renormalize)
    p = moe_permute(n, routed.expert_ids, w_ug.shape[0])
    h_buf, u = moe_gemm_up_swiglu_u(p.x_perm, p.offsets, w_ug)
    y_perm = moe_gemm_down(h_buf, p.offsets, w_down)
    y = moe_unpermute(y_perm, p.inv_map, routed.routing_w)
    after = dict(post_norm=post_norm, w_post=w_post, gate=gate, residual_scale=residual_scale, branch_scale=branch_scale,
                 next_norm=next_norm, w_next=w_next, eps=eps)
    r_out, n_out = moe_residual_norm(y, r, **after)
    return MoeLayer(r_out, n_out, routed, p, r, n, logits, rows, h_buf, u, y_perm, y, eps, after)


def moe_layer_backward(d_r_out: torch.Tensor | None, f: MoeLayer, w_norm, w_router: torch.Tensor, w_ug: torch.Tensor,
                       w_down: torch.Tensor, *, d_n_out=None, d_n_add=None, d_losses=None) -> dict:
    """Gradients of moe_layer_forward from those of its r_out, its n_out (in up to two parts) and its losses: dr in the
    stream's type; dw_router, dw_ug, dw_down bf16; dw_norm, dw_post, dw_next and d_gate fp32, None where there is none."""
    b = moe_residual_norm_backward(d_r_out, d_n_out, f.y, f.r_out, d_n_add=d_n_add, **f.after)
    e = moe_expert_backward(b.d_y, f.p, f.routed.routing_w, w_ug, w_down, f.h_buf, f.y_perm, f.u)
    d_logits = moe_router_backward(f.logits, f.routed, e["d_routing_w"], d_losses)
    dw_router = moe_grouped_wgrad(f.n, d_logits, f.rows, "out_in")[0]
    by_router = moe_grouped_dgrad(d_logits, f.rows, w_router[None], "out_in")
    dr, dw_norm = moe_rmsnorm_backward(e["dx"], f.r, w_norm, eps=f.eps, dy_add=by_router, dx_add=b.d_r)
    return {"dr": dr, "dw_norm": dw_norm, "dw_router": dw_router, "dw_ug": e["dw_ug"], "dw_down": e["dw_down"],
            "dw_post": b.d_w_post, "dw_next": b.d_w_next, "d_gate": b.d_gate, "d_logits": d_logits}


# ------------------------------------------------------------------ AdamW


class _AdamTensor(ctypes.Structure):
    _fields_ = [("n", _i64), ("offset", _i64), ("param_dtype", _i32), ("grad_dtype", _i32)]


class _AdamHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", _i64), ("seed", ctypes.c_uint32), ("stochastic", _i32)]


@dataclass
class Blocks8:
    """Moments in 8 bits: q uint8 [len] and a scale byte per 32 values, scales uint8 [len / 32]."""
    q: torch.Tensor
    scales: torch.Tensor


def _moment_places(params) -> tuple[list[int], int]:
    places, n = [], 0
    for p in params:
        places.append(n)
        n += (p.numel() + 31) // 32 * 32
    return places, n


@dataclass
class AdamW:
    """What AdamW keeps for a list of parameters: one buffer a moment, fp32 [len] or Blocks8 of len values, with tensor
    i's values from ``places[i]`` on (the sizes before it, each rounded up to 32), and with ``master`` a fp32 copy of
    the parameters at the same places. None of them may share memory. moe_adamw_state makes one."""
    params: list
    exp_avg: torch.Tensor | Blocks8
    exp_avg_sq: torch.Tensor | Blocks8
    master: torch.Tensor | None = None
    places: list = field(init=False, repr=False)
    len: int = field(init=False, repr=False)
    bits: int = field(init=False)

    def __post_init__(self):
        self.params = list(self.params)
        if not self.params:
            raise ValueError("no parameters")
        dev = self.params[0].device
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor) or p.dtype not in _LOGITS:
                raise TypeError(f"params[{i}] must be a bfloat16 or float32 tensor")
            _want(p, f"params[{i}]", p.dtype, tuple(p.shape), dev)
        self.places, self.len = _moment_places(self.params)
        self._device = dev
        self._moments = self._take_moments()
        self._want_apart(self._moments)
        count = len(self.params)
        self._table, self._hyper = (_AdamTensor * count)(), _AdamHyper()
        self._param_ptrs, self._grad_ptrs = (ctypes.c_uint64 * count)(), (ctypes.c_uint64 * count)()
        self._dtypes, self._shapes = [p.dtype for p in self.params], [p.shape for p in self.params]
        self._sizes, self._addresses = [p.numel() for p in self.params], [p.data_ptr() for p in self.params]
        self._param_ptrs[:] = self._addresses
        self._grad_dtypes = None
        for t, n, at, dtype in zip(self._table, self._sizes, self.places, self._dtypes):
            t.n, t.offset, t.param_dtype = n, at, _LOGITS[dtype]

    def _want_apart(self, moments):
        n, wide = self.len, 4 if self.bits == 32 else 1
        sizes = (wide * n, n // 32, wide * n, n // 32, 4 * n)
        spans = [(p.data_ptr(), p.numel() * p.element_size()) for p in self.params]
        spans += [(at, size) for at, size in zip(moments, sizes) if at is not None]
        spans = sorted((at, at + size) for at, size in spans if size)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("parameters, moments or the master share memory: each value is stepped once")

    def _take_moments(self):
        """Addresses of the moments, their scales and the master, checked at every step: a state that is read back may
        bring its own."""
        m, v, dev, n = self.exp_avg, self.exp_avg_sq, self._device, self.len
        self.bits = 8 if isinstance(m, Blocks8) else 32
        master = None if self.master is None else _want(self.master, "master", torch.float32, (n,), dev).data_ptr()
        if self.bits == 32:
            return (_want(m, "exp_avg", torch.float32, (n,), dev).data_ptr(), None,
                    _want(v, "exp_avg_sq", torch.float32, (n,), dev).data_ptr(), None, master)
        if not isinstance(v, Blocks8):
            raise TypeError("exp_avg_sq must be a Blocks8 as exp_avg is")
        return (_want(m.q, "exp_avg.q", torch.uint8, (n,), dev).data_ptr(),
                _want(m.scales, "exp_avg.scales", torch.uint8, (n // 32,), dev).data_ptr(),
                _want(v.q, "exp_avg_sq.q", torch.uint8, (n,), dev).data_ptr(),
                _want(v.scales, "exp_avg_sq.scales", torch.uint8, (n // 32,), dev).data_ptr(), master)

    def _take_params(self):
        """The parameters' addresses into their table; returns the moments'. Where a value stands follows from address, size,
        type and contiguity; if any of them has changed, all is checked again."""
        params, moments = self.params, self._take_moments()
        addresses = list(map(_Tensor.data_ptr, params))
        if (addresses != self._addresses or list(map(_Tensor.numel, params)) != self._sizes
                or [p.dtype for p in params] != self._dtypes or False in map(_Tensor.is_contiguous, params)
                or moments != self._moments):
            if len(params) != len(self._sizes):
                raise ValueError(f"the state is of {len(self._sizes)} parameters, not {len(params)}")
            for i, (p, dtype, shape) in enumerate(zip(params, self._dtypes, self._shapes)):
                _want(p, f"params[{i}]", dtype, tuple(shape), self._device)
            self._want_apart(moments)
            self._param_ptrs[:] = self._addresses = addresses
            self._moments = moments
        return moments

    def _take_grads(self, grads):
        if len(grads) != len(self._sizes):
            raise ValueError(f"{len(self._sizes)} parameters but {len(grads)} gradients")
        try:
            addresses = list(map(_Tensor.data_ptr, grads))
        except TypeError:
            i = next(i for i, g in enumerate(grads) if not isinstance(g, _Tensor))
            raise TypeError(f"grads[{i}] must be a torch.Tensor") from None
        dtypes = [g.dtype for g in grads]
        if dtypes != self._grad_dtypes:
            for i, dtype in enumerate(dtypes):
                if dtype not in _LOGITS:
                    raise TypeError(f"grads[{i}] must be bfloat16 or float32, got {dtype}")
            for t, dtype in zip(self._table, dtypes):
                t.grad_dtype = _LOGITS[dtype]
            self._grad_dtypes = dtypes
        index = self._device.index
        if (list(map(_Tensor.size, grads)) != self._shapes or list(map(_Tensor.get_device, grads)) != [index] * len(grads)
                or False in map(_Tensor.is_contiguous, grads)):
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):  # (names the one that does not fit)
                _want(g, f"grads[{i}]", g.dtype, tuple(shape), self._device)
        self._grad_ptrs[:] = addresses


def moe_adamw_state(params, *, bits: int = 32, master: bool = False) -> AdamW:
    """Zero moments in 32 or 8 bits for a list of parameters, and with ``master`` a fp32 copy of them, which the steps
    then read and write besides the parameters."""
    params = list(params)
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    if not params:
        raise ValueError("no parameters")
    dev = params[0].device
    places, n = _moment_places(params)

    def zeros():
        if bits == 32:
            return torch.zeros(n, device=dev)
        return Blocks8(torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(n // 32, dtype=torch.uint8, device=dev))

    copy = None
    if master:
        copy = torch.zeros(n, device=dev)
        for p, at in zip(params, places):
            copy[at:at + p.numel()] = p.detach().reshape(-1)
    return AdamW(params, zeros(), zeros(), copy)


def _device_scalar(v, name: str, dtype: torch.dtype, device):
    """The pointer of a one-value tensor."""
    return _want(v, name, dtype, (1,), device).data_ptr()


def moe_adamw_step(state: AdamW, grads, *, lr, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, step=1,
                   grad_scale: torch.Tensor | None = None, seed: int | None = None) -> None:
    """One AdamW step of ``state.params`` in place, a launch per 80 tensors. ``step`` counts from 1. ``lr`` may be a
    number or a fp32 [1] tensor on the device, ``step`` an int or an int32 [1] tensor, for steps captured in a graph;
    ``grad_scale`` fp32 [1] is multiplied to the gradients (a clipping factor). A ``seed`` rounds the second moment in 8
    bits, and bf16 parameters without a master, at random in proportion; without one they round to nearest."""
    m, ms, v, vs, master = state._take_params()
    state._take_grads(grads)
    dev, h = state._device, state._hyper
    lr_ptr = step_ptr = None
    if isinstance(lr, _Tensor):
        lr_ptr, lr = _device_scalar(lr, "lr", torch.float32, dev), 0.0
    if isinstance(step, _Tensor):
        step_ptr, step = _device_scalar(step, "step", torch.int32, dev), 1
    if grad_scale is not None:
        grad_scale = _device_scalar(grad_scale, "grad_scale", torch.float32, dev)
    if seed is not None and not 0 <= seed < 1 << 32:
        raise ValueError("seed must fit 32 bits")
    h.lr, (h.beta1, h.beta2), h.eps, h.weight_decay, h.step = lr, betas, eps, weight_decay, step
    h.seed, h.stochastic = (0, 0) if seed is None else (seed, 1)
    _check(load_library().moe_adamw_step(ctypes.addressof(state._table), ctypes.addressof(state._param_ptrs),
                                         ctypes.addressof(state._grad_ptrs), len(state._sizes), state.bits, state.len, m,
                                         ms, v, vs, master, ctypes.addressof(h), lr_ptr, step_ptr, grad_scale,
                                         _stream(state.params[0])), "moe_adamw_step")


def moe_adamw_moments(state: AdamW, *, exp_avg=None, exp_avg_sq=None):
    """The values of both moments, [len]: the fp32 buffers themselves, or bf16 of 8-bit ones (one launch)."""
    m, ms, v, vs, _ = state._take_moments()
    if state.bits == 32:
        return state.exp_avg, state.exp_avg_sq
    dev = state._device
    exp_avg = _out(exp_avg, "exp_avg", torch.bfloat16, (state.len,), dev)
    exp_avg_sq = _out(exp_avg_sq, "exp_avg_sq", torch.bfloat16, (state.len,), dev)
    _check(load_library().moe_adamw_moments(m, ms, v, vs, state.len, exp_avg.data_ptr(), exp_avg_sq.data_ptr(),
                                            _stream(exp_avg)), "moe_adamw_moments")
    return exp_avg, exp_avg_sq


__all__ = [
    "LIB_PATH", "MAX_EXPERTS", "MoeError", "Permuted", "grouped_swiglu_expert", "header_functions", "load_library",
    "grouped_swiglu_expert_gather", "moe_expert_forward", "moe_gemm_down", "moe_gemm_up_swiglu",
    "moe_gemm_up_swiglu_gather", "moe_gemm_up_swiglu_u", "moe_permute", "moe_permute_noalloc", "moe_unpermute",
    "permute_workspace_bytes", "W_LAYOUTS", "moe_grouped_dgrad", "moe_grouped_wgrad", "moe_permute_backward", "wgrad_workspace_bytes",
    "moe_grouped_projection", "moe_swiglu_backward", "moe_expert_backward",
    "moe_unpermute_backward",
    "ROUTER_MAX_TOPK", "Routed", "moe_router_topk", "moe_router_topk_losses", "moe_router_backward",
    "router_workspace_bytes", "Mxfp4", "mxfp4_row_bytes", "mxfp4_scale_bytes", "moe_mxfp4_quantize",
    "moe_mxfp4_quantize_weights", "moe_mxfp4_dequantize", "moe_grouped_projection_mxfp4", "moe_gemm_up_swiglu_mxfp4",
    "moe_gemm_up_swiglu_mxfp4_q", "moe_expert_forward_mxfp4",
    "Int4", "INT4_GROUPS", "moe_int4_quantize_weights", "moe_int4_dequantize_weights", "moe_grouped_projection_int4",
    "moe_gemm_up_swiglu_int4", "moe_expert_forward_int4",
    "NORM_MAX_WIDTH", "ResidualNormGrads", "moe_rmsnorm", "moe_rmsnorm_backward", "moe_residual_norm",
    "moe_residual_norm_backward", "norm_workspace_bytes", "MoeLayer", "moe_layer_forward", "moe_layer_backward",
    "AdamW", "Blocks8", "moe_adamw_state", "moe_adamw_step", "moe_adamw_moments",
]
