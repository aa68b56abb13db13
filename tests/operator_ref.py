"""Plain references of the operators between the ternary products (RMSNorm
with the residual, expert sorting and back, the dense int8 product), in numpy,
64 bits unless a step is defined as one fp32 rounding.  They share no code
with the library."""
from __future__ import annotations

import numpy as np

U24 = 2.0 ** -24        # half a step of fp32, relative
U8 = 2.0 ** -8          # half a step of bf16, relative


def bf16(a):
    """fp32 values rounded to bf16 (nearest even), as fp32.  Finite input."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32).reshape(np.shape(a))


def norm_exact(x, res, w, eps):
    """(h, n) of the formula in 64 bits."""
    h = x.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, h * r * w.astype(np.float64)


def norm_steps(x, res, w, eps):
    """(h, n) by the defined fp32 steps; the sum of squares in 64 bits."""
    f = np.float32
    h = x.astype(f) if res is None else (x.astype(f) + res.astype(f)).astype(f)
    h64 = h.astype(np.float64)
    mean = (np.sum(h64 * h64, axis=1, keepdims=True) / h.shape[1]).astype(f)
    r = (f(1) / np.sqrt(mean + f(eps), dtype=f)).astype(f)
    return h, ((h * r).astype(f) * w.astype(f)).astype(f)


def quant_steps(n):
    """The per-token int8 rule on fp32 rows: (codes, scales)."""
    f = np.float32
    a = np.max(np.abs(n), axis=1)
    inv = np.divide(f(127), a, out=np.zeros_like(a), where=a > 0)
    q = np.clip(np.rint((n * inv[:, None]).astype(f)), -127, 127).astype(np.int8)
    return q, (a / f(127)).astype(f)


def dispatch(ids, n_experts):
    """(rows, pairs, offsets) of the sorted pairs, one pair at a time."""
    T, k = ids.shape
    rows = np.full((T, k), -1, np.int32)
    pairs = np.full(T * k, -1, np.int32)
    offsets = np.zeros(n_experts + 1, np.int32)
    at = 0
    for e in range(n_experts):
        offsets[e] = at
        for p in np.flatnonzero(ids.reshape(-1) == e):
            rows.reshape(-1)[p] = at
            pairs[at] = p
            at += 1
    offsets[n_experts] = at
    return rows, pairs, offsets


def combine(rows, weights, ys):
    """(y, sum of magnitudes) in 64 bits."""
    T, k = rows.shape
    y = np.zeros((T, ys.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < ys.shape[0]:
                v = ys[rows[t, j]].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_grad(rows, weights, dy, ys):
    """(d_ys, written rows, d_weights, their sums of magnitudes) in 64 bits."""
    T, k = rows.shape
    d_ys = np.zeros(ys.shape)
    written = np.zeros(ys.shape[0], bool)
    d_w, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        g = dy[t].astype(np.float64)
        for j in range(k):
            r = rows[t, j]
            if 0 <= r < ys.shape[0]:
                d_ys[r] = g * (1.0 if weights is None else float(weights[t, j]))
                written[r] = True
                d_w[t, j] = np.sum(g * ys[r].astype(np.float64))
                mag[t, j] = np.sum(np.abs(g * ys[r].astype(np.float64)))
    return d_ys, written, d_w, mag


def dense_i8(xq, xs, wq, ws):
    """The product by its definition: exact integer sums (as 64-bit floating
    sums, which hold them exactly below 2^53), then two fp32 products."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    c = (xs.astype(np.float32)[:, None] * ws.astype(np.float32)[None, :]).astype(np.float32)
    return (acc.astype(np.float32) * c).astype(np.float32)
