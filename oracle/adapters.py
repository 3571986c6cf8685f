"""Oracle of the low-rank adapters: float64 definitions, one adapter at a time,
and the bounds that fp32 sums, the split of the low-rank values into three 16-bit
numbers and the final rounding put on a result. Test infrastructure only;
shares nothing with the library."""

from __future__ import annotations

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
LEAST = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}  # half of the smallest step (bf16, fp32: out of reach here)
U32 = 2.0 ** -24


def _split(kind: str, u: np.ndarray, largest) -> np.ndarray:
    """What three 16-bit numbers leave out of u: nothing of fp32's 24 bits (2^-24 for u's own rounding); fp16, brought to
    a largest of 2^13..2^14, half of its smallest step, 2^-25."""
    return np.abs(u) * U32 + (0.0 if kind == "bf16" else 2.0 ** -38 * largest)


def _rows(index, n):
    return [np.flatnonzero(index == i) for i in range(n)]


def adapt(y, x, a, b, index, scale=None):
    """``y [M, V]`` and so on in float64."""
    out = np.array(y, dtype=np.float64)
    for i, rows in enumerate(_rows(index, a.shape[0])):
        s = 1.0 if scale is None else scale[i]
        out[rows] += s * (x[rows] @ a[i].T) @ b[i].T
    return out


def adapt_bound(y, x, a, b, index, scale, kind):
    want, bound = adapt(y, x, a, b, index, scale), np.zeros(y.shape)
    hidden, rank = x.shape[1], a.shape[1]
    for i, rows in enumerate(_rows(index, a.shape[0])):
        s = 1.0 if scale is None else scale[i]
        u = s * (x[rows] @ a[i].T)
        du = (hidden + 64) * U32 * abs(s) * (np.abs(x[rows]) @ np.abs(a[i]).T)
        largest = np.abs(u).max(axis=1, keepdims=True, initial=0.0)
        lost = du + _split(kind, u, largest) + 2 * U32 * np.abs(u)
        inner = (lost + (2 * rank + 8) * U32 * np.abs(u)) @ np.abs(b[i]).T + U32 * np.abs(want[rows])
        bound[rows] = inner + HALF_STEP[kind] * (np.abs(want[rows]) + inner) + LEAST[kind]
    return want, bound


def adapt_grad(dy, x, a, b, index, scale=None):
    """``(dx, da, db)`` in float64."""
    dx, da, db = np.zeros(x.shape), np.zeros(a.shape), np.zeros(b.shape)
    for i, rows in enumerate(_rows(index, a.shape[0])):
        s = 1.0 if scale is None else scale[i]
        g, u = s * (dy[rows] @ b[i]), s * (x[rows] @ a[i].T)
        dx[rows], da[i], db[i] = g @ a[i], g.T @ x[rows], dy[rows].T @ u
    return dx, da, db


def adapt_grad_bound(dy, x, a, b, index, scale, kind, out):
    """``(want, bound)`` of each; ``out``: da's and db's type."""
    wants = adapt_grad(dy, x, a, b, index, scale)
    dx, da, db = (np.zeros(t.shape) for t in wants)
    m, rank, n = x.shape[0], a.shape[1], a.shape[0]
    parts = []
    for i, rows in enumerate(_rows(index, n)):
        s = 1.0 if scale is None else scale[i]
        g, u = s * (dy[rows] @ b[i]), s * (x[rows] @ a[i].T)
        eg = (dy.shape[1] + 64) * U32 * abs(s) * (np.abs(dy[rows]) @ np.abs(b[i])) + 2 * U32 * np.abs(g)
        eu = (x.shape[1] + 64) * U32 * abs(s) * (np.abs(x[rows]) @ np.abs(a[i]).T) + 2 * U32 * np.abs(u)
        parts.append((i, rows, g, u, eg, eu))
    for i, rows, g, u, eg, eu in parts:
        row = np.abs(g).max(axis=1, keepdims=True, initial=0.0)
        dx[rows] = (eg + _split(kind, g, row) + (2 * rank + 8) * U32 * np.abs(g)) @ np.abs(a[i])
        da[i] = (eg + _split(kind, g, np.abs(g).max(initial=0.0)) + (2 * m + 8) * U32 * np.abs(g)).T @ np.abs(x[rows])
        db[i] = np.abs(dy[rows]).T @ (eu + _split(kind, u, np.abs(u).max(initial=0.0)) + (2 * m + 8) * U32 * np.abs(u))
    kinds = (kind, out, out)
    return wants, [e + HALF_STEP[k] * (np.abs(w) + e) + LEAST[k] for e, w, k in zip((dx, da, db), wants, kinds)]
