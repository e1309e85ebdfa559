"""The router in 64 bits: top-k, weights, losses and the gradient of the logits (test infrastructure only).

For a row x: lse = log sum exp(x), p = exp(x - lse). The chosen experts are those of the largest logits, lowest index
first among equals; -inf is never chosen (id -1, weight 0). Losses over the n rows that are not all -inf:
E sum_e f_e P_e with f_e = counts_e / sum counts and P the mean probabilities, and the mean of lse^2. The gradient is
written with softmax's Jacobian diag(p) - p p^T applied to dL/dp, term by term. Rows here hold no NaN and no +inf.
"""

from __future__ import annotations

import numpy as np


def softmax_rows(x) -> tuple[np.ndarray, np.ndarray]:
    """(p [T, E], lse [T]) of float64 logits; a row of -inf alone has p = 0 and lse = -inf."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max(axis=1)
    m0 = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(x - m0[:, None])
    s = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = m0 + np.log(s)
    return e / np.where(s > 0, s, 1.0)[:, None], lse


def topk(x, k: int, renormalize: bool):
    """(ids int32 [T, k], w float64 [T, k], lse float64 [T])."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    p, lse = softmax_rows(x)
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] != -np.inf), key=lambda e: (-x[t, e], e))[:k]
        ids[t, :len(order)] = order
        chosen = p[t, order]
        if renormalize and len(order):
            # a softmax over the chosen logits alone: the smallest ones underflow no earlier than there
            z = np.exp(x[t, order] - x[t, order[0]])
            chosen = z / z.sum()
        w[t, :len(order)] = chosen
    return ids, w, lse


def losses(x, ids):
    """(counts int32 [E], n, P float64 [E], [balance, z])."""
    x = np.asarray(x, dtype=np.float64)
    E = x.shape[1]
    p, lse = softmax_rows(x)
    live = ~np.isneginf(lse)
    n = int(live.sum())
    counts = np.bincount(ids[ids >= 0], minlength=E)
    f = counts / max(1, counts.sum())
    P = p[live].sum(axis=0) / max(1, n)
    z = float((lse[live] ** 2).sum()) / max(1, n)
    return counts.astype(np.int32), n, P, np.array([E * float((f * P).sum()), z])


def backward(x, ids, renormalize: bool, d_w=None, d_losses=None, counts=None, n=None):
    """(d_logits float64 [T, E], the sum of the magnitudes of the terms each element is made of)."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    p, lse = softmax_rows(x)
    d = np.zeros((T, E))
    size = np.zeros((T, E))
    f = None
    if d_losses is not None:
        f = counts / max(1, counts.sum())
    for t in range(T):
        if np.isneginf(lse[t]):
            continue
        dp = np.zeros(E)  # dL/dp
        mag = np.zeros(E)
        if d_losses is not None:
            dp += d_losses[0] * E * f / max(1, n)
            mag += np.abs(dp)
            dz = 2 * d_losses[1] * lse[t] / max(1, n)
            d[t] += dz * p[t]
            size[t] += np.abs(dz) * p[t]
        if d_w is not None:
            kept = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
            sel = ids[t, kept]
            if renormalize:
                z = np.exp(x[t, sel] - x[t, sel].max()) if len(kept) else np.zeros(0)
                w = z / z.sum() if len(kept) else z
                g = d_w[t, kept].astype(np.float64)
                for j, e in enumerate(sel):
                    d[t, e] += w[j] * (g[j] - (g * w).sum())
                    size[t, e] += w[j] * (abs(g[j]) + (np.abs(g) * w).sum())
            else:
                for j, e in zip(kept, sel):
                    dp[e] += d_w[t, j]
                    mag[e] += abs(float(d_w[t, j]))
        d[t] += p[t] * (dp - (p[t] * dp).sum())
        size[t] += p[t] * (mag + (p[t] * mag).sum())
    return d, size
