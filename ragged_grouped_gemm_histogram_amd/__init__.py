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
import os
import re
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_grouped.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_grouped.h")
MAX_EXPERTS = 1024

MOE_OK = 0

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
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
]
