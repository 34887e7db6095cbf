"""Low-rank adapters per token and their gradients, float64 (oracle; test
infrastructure)."""

from __future__ import annotations

import numpy as np


def forward(x, a, b, ids, y=None, scaling=None):
    """(out, u): u[t] = A[id] x[t], out[t] = y[t] + s[id] B[id] u[t]."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    T, (L, N, R) = x.shape[0], b.shape
    out = np.zeros((T, N)) if y is None else np.array(y, np.float64)
    u = np.zeros((T, R))
    for t in range(T):
        k = int(ids[t])
        if 0 <= k < L:
            u[t] = a[k] @ x[t]
            out[t] += (1.0 if scaling is None else float(scaling[k])) * (b[k] @ u[t])
    return out, u


def backward(dy, x, a, b, ids, u, dx_base=None, scaling=None):
    """(dx, dA, dB, d), d[t] = B[id]^T dy[t]."""
    dy, x, a, b, u = (np.asarray(v, np.float64) for v in (dy, x, a, b, u))
    T, (L, N, R) = x.shape[0], b.shape
    dx = np.zeros_like(x) if dx_base is None else np.array(dx_base, np.float64)
    da, db, d = np.zeros_like(a), np.zeros_like(b), np.zeros((T, R))
    for t in range(T):
        k = int(ids[t])
        if 0 <= k < L:
            s = 1.0 if scaling is None else float(scaling[k])
            d[t] = b[k].T @ dy[t]
            dx[t] += s * (a[k].T @ d[t])
            da[k] += s * np.outer(d[t], x[t])
            db[k] += s * np.outer(dy[t], u[t])
    return dx, da, db, d
