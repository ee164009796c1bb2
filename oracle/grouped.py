"""fp64 oracle of the layer's separate operators (``include/moe.h``): the
grouped expert products and their gradients, 8-bit row codes, the 8-bit
product, and the combine with its gradients.  Plain NumPy loops over rows and
experts; no code shared with the GPU path."""
from __future__ import annotations

import numpy as np


def segments(offsets, counts, rows, E):
    """(begin, end) of each expert's rows, cut to [0, rows)."""
    out = []
    for e in range(E):
        b = int(offsets[e])
        n = int(counts[e]) if counts is not None else int(offsets[e + 1]) - b
        end = b + max(n, 0)
        lo = min(max(b, 0), rows)
        out.append((lo, max(lo, min(end, rows))))
    return out


def lookup(x, row_ids, row_div, rows):
    """The rows of x in sorted order [rows, K]; rows that stand for zeros are zero."""
    x = np.asarray(x, dtype=np.float64)
    if row_ids is None:
        return x
    out = np.zeros((rows, x.shape[1]))
    for r in range(rows):
        i = int(row_ids[r])
        if i >= 0 and i // row_div < x.shape[0]:
            out[r] = x[i // row_div]
    return out


def grouped_matmul(xs, segs, w):
    """y [rows, N] for looked-up rows xs [rows, K]; NaN in rows of no segment."""
    y = np.full((xs.shape[0], w.shape[1]), np.nan)
    for e, (a, b) in enumerate(segs):
        if b > a:
            y[a:b] = xs[a:b] @ np.asarray(w[e], dtype=np.float64).T
    return y


def grouped_matmul_backward(dy, xs, segs, w):
    """(dx [rows, K], NaN in rows of no segment; dw [E, N, K])."""
    E, N, K = w.shape
    dx, dw = np.full((dy.shape[0], K), np.nan), np.zeros((E, N, K))
    for e, (a, b) in enumerate(segs):
        if b > a:
            dx[a:b] = dy[a:b] @ np.asarray(w[e], dtype=np.float64)
            dw[e] = dy[a:b].T @ xs[a:b]
    return dx, dw


def quantize_rows(x):
    """(codes int64, scale float32) of each row of a float32-valued matrix."""
    x = np.asarray(x, dtype=np.float64)
    q, s = np.zeros(x.shape, dtype=np.int64), np.zeros(x.shape[0], dtype=np.float32)
    for r in range(x.shape[0]):
        if not np.isfinite(x[r]).all():
            s[r] = np.nan
            continue
        s[r] = np.float32(np.abs(x[r]).max() / 127.0)
        if s[r] > 0:
            q[r] = np.clip(np.rint(x[r] / np.float64(s[r])), -127, 127).astype(np.int64)
    return q, s


def grouped_matmul_i8(q, scale, row_ids, row_div, segs, wq, w_scale, rows):
    """y [rows, N] of 8-bit codes; NaN in rows of no segment."""
    y = np.full((rows, wq.shape[1]), np.nan)
    for e, (a, b) in enumerate(segs):
        for r in range(a, b):
            i = r if row_ids is None else int(row_ids[r])
            src = i if row_ids is None else i // row_div
            if i < 0 or src >= q.shape[0]:
                y[r] = 0.0
                continue
            acc = wq[e].astype(np.int64) @ q[src].astype(np.int64)
            y[r] = acc.astype(np.float64) * np.float64(scale[src]) * w_scale[e].astype(np.float64)
    return y


def combine(y, inv, weights):
    """out [T, H]; an inv outside [0, rows) adds nothing."""
    T, k = inv.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < y.shape[0]:
                out[t] += (1.0 if weights is None else float(weights[t, j])) * y[inv[t, j]]
    return out


def combine_backward(dout, y, inv, weights):
    """(dy [rows, H], NaN in rows that no assignment names; dweights [T, k])."""
    T, k = inv.shape
    dy, dw = np.full(y.shape, np.nan), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = inv[t, j]
            if 0 <= p < y.shape[0]:
                dy[p] = (1.0 if weights is None else float(weights[t, j])) * dout[t]
                dw[t, j] = dout[t] @ y[p]
    return dy, dw
