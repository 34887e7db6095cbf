"""A mixture of experts: the router, products grouped by expert with their
gradients and the sum of the experts' results, float64 (oracle; test
infrastructure)."""

from __future__ import annotations

import numpy as np

from . import formats as F
from .checkpoint import keep, values


def route(logits, k, renormalize):
    """(weights, ids): per token the k largest logits, ties to the lowest
    index, never minus infinity or NaN (id -1, weight 0)."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-l[t, e], e))[:k]
        order = [e for e in order if l[t, e] > -np.inf]
        if not order:
            continue
        top = l[t, order[0]]
        w = np.exp(l[t, order] - top)
        weights[t, :len(order)] = w / (w.sum() if renormalize else np.exp(l[t] - top).sum())
        ids[t, :len(order)] = order
    return weights, ids


def layout(ids, E):
    """(offsets, rows, slots) of the (token, choice) pairs by expert."""
    T, k = ids.shape
    rows, slots, offsets = np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32), [0]
    for e in range(E):
        pairs = [(t, j) for t, j in np.argwhere(ids == e)]
        for i, (t, j) in enumerate(pairs):
            slots[t, j] = offsets[-1] + i
            rows[offsets[-1] + i] = t
        offsets.append(offsets[-1] + len(pairs))
    return np.array(offsets, np.int32), rows, slots


def route_backward(d_weights, logits, ids, weights, renormalize):
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    dw, w = np.asarray(d_weights, np.float64), np.asarray(weights, np.float64)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        used = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < l.shape[1]]
        mean = sum(w[t, j] * dw[t, j] for j in used)
        if not renormalize and l[t].max() > -np.inf:
            p = np.exp(l[t] - l[t].max())
            out[t] = -mean * p / p.sum()
        for j in used:
            out[t, ids[t, j]] += w[t, j] * (dw[t, j] - (mean if renormalize else 0.0))
    return out


def segments(offsets, S):
    """(expert, slice) of the segments, as the library clamps them."""
    for e in range(len(offsets) - 1):
        lo = min(max(int(offsets[e]), 0), S)
        hi = min(max(int(offsets[e + 1]), lo), S)
        if hi > lo:
            yield e, slice(lo, hi)


def gemm(x, w, offsets, rows, S):
    """(y, sum of magnitudes) from the operands' values x [X, K], w [E, N, K];
    NaN where no segment is."""
    y = np.full((S, w.shape[1]), np.nan)
    mag = np.full_like(y, np.nan)
    rows = np.arange(S) if rows is None else rows
    for e, at in segments(offsets, S):
        y[at] = x[rows[at]] @ w[e].T
        mag[at] = np.abs(x[rows[at]]) @ np.abs(w[e]).T
    return y, mag


def mx_values(codes, scales, code):
    """What MXFP8 codes [.., K] with scale bytes [.., K / 32] stand for."""
    v = F.decode(codes, code).astype(np.float64).reshape(scales.shape + (32,))
    return (v * np.exp2(scales.astype(np.float64) - 127)[..., None]).reshape(codes.shape)


def mx_rows(x, code):
    """Rows quantized in blocks of 32 (the last may be shorter), as values."""
    n = x.shape[-1]
    full = np.concatenate([x, np.zeros((x.shape[0], -n % 32), x.dtype)], 1)
    return values(*keep(full, code, "ue8m0"), code)[:, :n].astype(np.float64)


def backward(dY, W, X, offsets, rows, code):
    """(dX, dW, magnitudes of both) from binary32 arrays of bfloat16 values."""
    S, (E, N, K) = dY.shape[0], W.shape
    dX, dW = np.full((S, K), np.nan), np.zeros((E, N, K))
    mX, mW = np.full((S, K), np.nan), np.zeros((E, N, K))
    rows = np.arange(S) if rows is None else rows
    dyn = mx_rows(dY, code)
    for e, at in segments(offsets, S):
        wt = mx_rows(np.ascontiguousarray(W[e].T), code)  # [K, N]
        dX[at], mX[at] = dyn[at] @ wt.T, np.abs(dyn[at]) @ np.abs(wt).T
        dyt = mx_rows(np.ascontiguousarray(dY[at].T), code)
        xt = mx_rows(np.ascontiguousarray(X[rows[at]].T), code)
        dW[e], mW[e] = dyt @ xt.T, np.abs(dyt) @ np.abs(xt).T
    return dX, dW, mX, mW


def combine(y, slots, weights):
    """(out, sum of magnitudes)."""
    y = np.asarray(y, np.float64)
    T, k = slots.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                term = (1.0 if weights is None else float(weights[t, j])) * y[slots[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_backward(d_out, y, slots, weights):
    """(dy, d_weights, magnitudes of d_weights); dy NaN where no pair is."""
    d, y = np.asarray(d_out, np.float64), np.asarray(y, np.float64)
    dy, dw = np.full_like(y, np.nan), np.zeros(slots.shape)
    mag = np.zeros(slots.shape)
    for t, j in np.ndindex(*slots.shape):
        s = slots[t, j]
        if 0 <= s < y.shape[0]:
            dy[s] = (1.0 if weights is None else float(weights[t, j])) * d[t]
            dw[t, j], mag[t, j] = d[t] @ y[s], np.abs(d[t]) @ np.abs(y[s])
    return dy, dw, mag
