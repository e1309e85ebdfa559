"""4-bit weights with group scales, W = s (q - z): rounding, values and products in 64 bits (test infrastructure only)."""

from __future__ import annotations

import numpy as np

from .bf16 import bf16_bits_to_f64, f64_to_bf16_bits


def quantize(w, group: int, symmetric: bool):
    """(q uint8 [N, K] of one code each, scales bf16 bits [G, N], zeros uint8 [G, N] or None) of float32 weights [N, K]."""
    N, K = w.shape
    G = -(-K // group)
    q, s = np.zeros((N, K), np.uint8), np.zeros((G, N), np.uint16)
    z = None if symmetric else np.zeros((G, N), np.uint8)
    f = np.float32
    for j in range(G):
        part = w[:, j * group:(j + 1) * group].astype(f)
        bad = ~np.isfinite(part).all(1)
        clean = np.where(bad[:, None], f(0), part)
        lo, hi = np.minimum(clean.min(1), f(0)), np.maximum(clean.max(1), f(0))
        with np.errstate(over="ignore"):
            width = hi - lo
        bad |= ~np.isfinite(width)
        scale = np.maximum(-lo, hi) / f(7) if symmetric else width / f(15)
        s[j] = np.where(bad, 0x7FC0, f64_to_bf16_bits(np.where(bad, f(0), scale).astype(f)))
        step = bf16_bits_to_f64(np.where(bad, 0, s[j]).astype(np.uint16)).astype(f)
        step = np.where(step > 0, step, f(1)).astype(f)
        zero = np.full(N, f(8)) if symmetric else np.clip(np.rint(-lo / step), 0, 15).astype(f)
        code = np.clip(np.rint(clean / step[:, None]) + zero[:, None], 0, 15)
        q[:, j * group:(j + 1) * group] = np.where(bad[:, None], 8, code)
        if not symmetric:
            z[j] = np.where(bad, 0, zero)
    return q, s, z


def pack(q):
    """[N, K] codes to [N, 16 * ceil(K / 32)] bytes, the even value in the low half."""
    N, K = q.shape
    full = np.zeros((N, 32 * -(-K // 32)), np.uint8)
    full[:, :K] = q
    return full[:, 0::2] | (full[:, 1::2] << 4)


def unpack(packed, K: int):
    q = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    q[:, 0::2], q[:, 1::2] = packed & 15, packed >> 4
    return q[:, :K]


def values(q, scales, zeros, group: int):
    """(float64 [N, K] weights, and s (16 + q), s (16 + z): what the kernel's sums are made of)"""
    K = q.shape[1]
    at = np.arange(K) // group
    s = bf16_bits_to_f64(scales).T[:, at]
    z = 8.0 if zeros is None else zeros.astype(np.float64).T[:, at]
    return s * (q - z), np.abs(s) * (32.0 + q + z)
