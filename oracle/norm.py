"""Norms around a block in 64 bits, forward and backward (test infrastructure only).

With rs(x) = 1 / sqrt(mean(x^2) + eps): u = y rs(y) w_post (or y), r' = a r + b gate u, n = r' rs(r') w_next. Each call
also gives, element by element, the sum of the magnitudes of the terms a result is made of: what fp32 errors scale with.
The gradient is written from the Jacobian of x -> x rs(x), rs (I - x x^T rs^2 / d), as a matrix.
"""

from __future__ import annotations

import numpy as np


def rs(x, eps):
    return 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def forward(r, y=None, *, post=False, w_post=1.0, gate=1.0, a=1.0, b=1.0, nxt=True, w_next=1.0, eps=1e-6):
    """(r', n, magnitudes of r', magnitudes of n); n is None without the next norm."""
    x, mag = r, np.abs(r)
    if y is not None:
        u = y * rs(y, eps) * w_post if post else y
        x = a * r + b * gate * u
        mag = np.abs(a * r) + np.abs(b * gate * u)
    if not nxt:
        return x, None, mag, None
    s = rs(x, eps)
    return x, x * s * w_next, mag, mag * s * np.abs(w_next)


def through_norm(x, w, dn, eps):
    """Gradient of x (and magnitudes) and the terms of w's, row by row through the Jacobian."""
    T, d = x.shape
    s = rs(x, eps)
    h = dn * w
    dx, mag = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        J = s[t, 0] * (np.eye(d) - np.outer(x[t], x[t]) * (s[t, 0] ** 2 / d))
        dx[t] = J.T @ h[t]
        mag[t] = s[t, 0] * (np.abs(h[t]) + np.abs(x[t]) * s[t, 0] ** 2 * np.abs(h[t] * x[t]).mean())
    return dx, mag, dn * x * s


def through_wide_norm(x, w, dn, eps):
    """through_norm for rows whose d x d Jacobian would be too large: its product with h, written out."""
    s = rs(x, eps)
    h = dn * w
    dx = s * (h - x * s ** 2 * (h * x).mean(axis=1, keepdims=True))
    mag = s * (np.abs(h) + np.abs(x) * s ** 2 * np.abs(h * x).mean(axis=1, keepdims=True))
    return dx, mag, dn * x * s


def backward(d_r, d_n, r_out, y=None, *, post=False, w_post=1.0, gate=1.0, a=1.0, b=1.0, nxt=True, w_next=1.0, eps=1e-6,
             gate_kind="none", through=through_norm):
    """dict of name -> (gradient, magnitudes): r, and y, gate, w_post, w_next where there are any."""
    out = {}
    g = np.zeros_like(r_out) if d_r is None else d_r
    mag = np.abs(g)
    if nxt:
        dx, m, terms = through(r_out, w_next, d_n, eps)
        g, mag = g + dx, mag + m
        out["w_next"] = terms.sum(0), np.abs(terms).sum(0)
    out["r"] = a * g, abs(a) * mag
    if y is None:
        return out
    u = y * rs(y, eps) * w_post if post else y
    if gate_kind == "token":
        out["gate"] = b * (g * u).sum(1, keepdims=True), abs(b) * (mag * np.abs(u)).sum(1, keepdims=True)
    if gate_kind == "channel":
        out["gate"] = b * (g * u).sum(0), abs(b) * (mag * np.abs(u)).sum(0)
    du, m = b * gate * g, np.abs(b * gate) * mag
    if post:
        dy, my, terms = through(y, w_post, du, eps)
        s = rs(y, eps)
        out["w_post"] = terms.sum(0), (m * np.abs(y) * s).sum(0)
        w = np.abs(w_post)
        out["y"] = dy, s * (m * w + np.abs(y) * s ** 2 * (m * w * np.abs(y)).mean(1, keepdims=True))
    else:
        out["y"] = du, m
    return out
