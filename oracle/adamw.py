"""AdamW in 64 bits, and its 8-bit moments bit for bit (test infrastructure only).

The codes follow from fp32 moments taken in the order (m b1) + (g (1 - b1)) and (v b2) + ((g g) (1 - b2)), each operation
rounded, so NumPy's float32 gives them exactly. First moment: float8 e4m3 by search among all 256 values, the block's
largest in [128, 256). Second: code c is (1 + (c % 8) / 8) 2^(c // 8), 0 for c = 0, the largest with c // 8 = 30.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def step64(p, g, m, v, *, lr, b1, b2, eps, wd, t):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    update = lr / (1 - b1 ** t) * m / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return (1 - lr * wd) * p - update, m, v, update


def moments32(g, m, v, b1, b2, scale=None):
    """fp32 moments, every operation rounded."""
    g = g.astype(F32) * F32(1.0 if scale is None else scale)
    return (m * F32(b1) + g * F32(1 - b1)).astype(F32), (v * F32(b2) + (g * g) * F32(1 - b2)).astype(F32)


def e4m3_values() -> np.ndarray:
    """The values of codes 0 .. 126 (not negative, finite)."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))


def e5m3_values() -> np.ndarray:
    c = np.arange(256)
    return np.where(c == 0, 0.0, (1 + (c & 7) / 8) * 2.0 ** (c >> 3))


def _blocks(x):
    b = np.asarray(x, dtype=F32).reshape(-1, 32).astype(np.float64)
    bad = ~np.isfinite(b).all(axis=1)
    top = np.abs(np.where(bad[:, None], 0.0, b)).max(axis=1)
    exponent = np.floor(np.log2(np.where(top > 0, top, 1.0))).astype(int)
    exponent = np.where(2.0 ** exponent > top, exponent - 1, exponent)
    exponent = np.where(2.0 ** (exponent + 1) <= top, exponent + 1, exponent)
    return b, bad, np.where(top > 0, exponent, -1000)


def to_e4m3(m):
    """(codes uint8 [n], scale bytes [n / 32])"""
    b, bad, exponent = _blocks(m)
    byte = np.maximum(exponent - 7 + 127, 1)
    y = np.where(bad[:, None], 0.0, b) * 2.0 ** (127.0 - byte)[:, None]
    grid = e4m3_values()
    mid = (grid[1:] + grid[:-1]) / 2
    low = np.searchsorted(mid, np.abs(y), side="left")  # a tie stays low ...
    tie = (low < len(mid)) & (np.abs(y) == mid[np.minimum(low, len(mid) - 1)])
    code = low + (tie & (low % 2 == 1))  # ... unless the one above is even
    code = code | (np.signbit(b) & ~bad[:, None]) * 128
    return code.astype(np.uint8).reshape(-1), np.where(bad, 255, byte).astype(np.uint8)


def of_e4m3(q, s):
    mag = np.append(e4m3_values(), np.nan)[(q & 127).reshape(-1, 32)]
    v = np.where((q & 128).reshape(-1, 32) != 0, -mag, mag) * 2.0 ** (s.astype(float) - 127)[:, None]
    return np.where((s == 255)[:, None], np.nan, v).reshape(-1)


def to_e5m3(v, random=None):
    """(codes, scale bytes); `random`: 16-bit integers, one a value, for rounding at random."""
    b, bad, exponent = _blocks(v)
    byte = np.maximum(exponent - 30 + 127, 1)
    y = np.where(bad[:, None], 0.0, b) * 2.0 ** (127.0 - byte)[:, None]
    grid = e5m3_values()
    low = np.clip(np.searchsorted(grid, y, side="right") - 1, 0, 254)  # the code at or below
    gap = grid[low + 1] - grid[low]
    part = (y - grid[low]) / gap
    if random is None:
        up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    else:  # the 20 dropped bits and 16 random ones above four zeros carry over
        up = np.floor(part * 2 ** 20) + random.reshape(-1, 32) * 16.0 >= 2 ** 20
    code = np.where(y > 0, np.maximum(low + (up & (low > 0)), 1), 0)
    return np.where(bad[:, None], 0, code).astype(np.uint8).reshape(-1), np.where(bad, 255, byte).astype(np.uint8)


def of_e5m3(q, s):
    v = e5m3_values()[q.reshape(-1, 32)] * 2.0 ** (s.astype(float) - 127)[:, None]
    return np.where((s == 255)[:, None], np.nan, v).reshape(-1)


def mix(h):
    h = np.asarray(h, dtype=np.uint64)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def random_bits(seed: int, step: int, places) -> np.ndarray:
    places = np.asarray(places, dtype=np.uint64)
    key = mix(np.uint64(seed) ^ mix(step))
    high = ((places >> np.uint64(32)) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    return mix(((places & np.uint64(0xFFFFFFFF)) + high + key) & np.uint64(0xFFFFFFFF)).astype(np.int64)
