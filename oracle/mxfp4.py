"""MXFP4 in 64 bits, from the format's definition (test infrastructure only).

OCP Microscaling Formats v1.0: 32 values share a scale 2^e with e = floor(log2(largest magnitude)) - 2 (2 is the
exponent of the largest 4-bit value, 6 = 1.5 * 2^2), stored as e + 127; values are E2M1. Here a value is rounded by
comparing it with every grid point, and halfway cases go to the even code.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(K: int) -> int:
    return 16 * -(-K // 32)


def scale_bytes(K: int) -> int:
    return 16 * -(-K // 512)


def nearest_code(y) -> np.ndarray:
    """Codes 0..7 of magnitudes y >= 0: the nearest grid value, the even code halfway, 7 past the end."""
    dist = np.abs(np.asarray(y, dtype=np.float64)[..., None] - GRID)
    near = dist.min(axis=-1, keepdims=True)
    tied = dist == near  # at most two neighbours
    codes = np.arange(8)
    even = np.where(tied & (codes % 2 == 0), codes, -1).max(axis=-1)
    return np.where(even >= 0, even, np.argmax(tied, axis=-1)).astype(np.uint8)


def quantize(x):
    """(q uint8 [R, row bytes], scales uint8 [R, scale bytes]) of float64 rows x [R, K]."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    n = -(-K // 32)
    b = np.zeros((R, n * 32))
    b[:, :K] = x
    b = b.reshape(R, n, 32)
    finite = np.isfinite(b).all(axis=-1)
    b = np.where(finite[..., None], b, 0.0)
    top = np.abs(b).max(axis=-1)
    _, ex = np.frexp(top)  # top = m 2^ex, m in [1/2, 1): floor(log2 top) = ex - 1
    e = np.where(top > 0, np.maximum(ex - 3, -127), -127)
    code = nearest_code(np.ldexp(np.abs(b), -e[..., None]))
    code |= (np.signbit(b).astype(np.uint8) << 3)
    flat = code.reshape(R, n * 32)
    q = flat[:, 0::2] | (flat[:, 1::2] << 4)
    scales = np.zeros((R, scale_bytes(K)), dtype=np.uint8)
    scales[:, :n] = np.where(finite, e + 127, 255)
    return q, scales


def dequantize(q, scales, K: int) -> np.ndarray:
    """float64 values [..., K]; NaN for a block whose scale byte is 255."""
    q = np.asarray(q, dtype=np.uint8)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    byte = np.repeat(np.asarray(scales)[..., :code.shape[-1] // 32].astype(np.int64), 32, axis=-1)
    with np.errstate(over="ignore"):
        v = np.where(byte == 255, np.nan, np.ldexp(v, byte - 127))
    return v[..., :K]
