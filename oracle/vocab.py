"""The vocabulary matrix's training operators in float64, straight from their
definitions: the lm_head's softmax cross entropy with its gradient, the
embedding lookup with its gradient, and the bounds that fp32 sums and 16-bit
roundings put on a result of the GPU's.

numpy only; shares no code with the HIP path.
"""

from __future__ import annotations

import numpy as np

# half a step of each type, relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
U32 = 2.0 ** -24


def kept_rows(labels: np.ndarray, vocab: int, ignore: int) -> np.ndarray:
    """Rows that count: neither left out nor labelled outside the vocabulary."""
    return np.flatnonzero((labels != ignore) & (labels >= 0) & (labels < vocab))


def head_xent(x, w, labels, vocab, ignore=-100, scale=1.0, z_weight=0.0):
    """(loss, lse): 0 for a row left out, NaN for a label outside."""
    m = x.shape[0]
    loss, lse = np.zeros(m), np.zeros(m)
    bad = (labels != ignore) & ~((labels >= 0) & (labels < vocab))
    loss[bad] = lse[bad] = np.nan
    for i in kept_rows(labels, vocab, ignore):
        z = scale * (w[:vocab] @ x[i])
        top = z.max()
        lse[i] = top + np.log(np.exp(z - top).sum())
        loss[i] = lse[i] - z[labels[i]] + z_weight * lse[i] ** 2
    return loss, lse


def head_xent_grad(x, w, labels, lse, grad, vocab, ignore=-100, scale=1.0, z_weight=0.0):
    """(dx, dw, d): d is [kept rows, vocab]."""
    kept = kept_rows(labels, vocab, ignore)
    d = np.zeros((len(kept), vocab))
    for p, i in enumerate(kept):
        z = scale * (w[:vocab] @ x[i])
        d[p] = (1 + 2 * z_weight * lse[i]) * np.exp(z - lse[i])
        d[p, labels[i]] -= 1
        d[p] *= scale * grad[i]
    dx = np.zeros(x.shape)
    dx[kept] = d @ w[:vocab]
    dw = np.zeros(w.shape)
    dw[:vocab] = d.T @ x[kept]
    return dx, dw, d


def embed(tokens, w, scale=1.0):
    out = np.zeros((len(tokens), w.shape[1]))
    for j, t in enumerate(tokens):
        if 0 <= t < w.shape[0]:
            out[j] = scale * w[t]
    return out


def embed_grad(tokens, dy, rows, scale=1.0):
    dw = np.zeros((rows, dy.shape[1]))
    for j, t in enumerate(tokens):
        if 0 <= t < rows:
            dw[t] += scale * dy[j]
    return dw


# -- bounds ------------------------------------------------------------------


def logit_bound(x, w, kept, vocab, scale):
    """Per row, how far a logit may be off: hidden products summed in fp32 in
    an order the matrix cores do not specify (2 * hidden * 2^-24 of the sum of
    magnitudes) and the two factors of the base-2 logit."""
    mag = np.abs(x[kept]) @ np.abs(w[:vocab]).T * abs(scale)
    return ((2.0 * x.shape[1] + 4.0) * U32 * mag).max(axis=1, initial=0.0)


def lse_bound(x, w, kept, vocab, scale, lse):
    """Logits, then a sum of exponentials whose longest chain has 16 terms of a
    lane, 4 joins, the tiles a thread merges and 16 merges, each with an
    exponential of 2 ulp, and the roundings of the result."""
    tiles = -(-vocab // 256)
    chain = 16 + 4 + 2 * -(-tiles // 16) + 2 * 16 + 8
    return logit_bound(x, w, kept, vocab, scale) + 2.0 * chain * U32 + 8.0 * U32 * np.abs(lse[kept])


def loss_bound(x, w, kept, vocab, scale, z_weight, lse):
    b = lse_bound(x, w, kept, vocab, scale, lse)
    top = np.abs(lse[kept]) + b
    return (2.0 * b + 2.0 * abs(z_weight) * top * b + 8.0 * U32 * (top + abs(z_weight) * top ** 2)
            + 4.0 * U32 * scale_mag(x, w, kept, vocab, scale))


def scale_mag(x, w, kept, vocab, scale):
    return np.abs(scale * (x[kept] @ w[:vocab].T)).max(axis=1, initial=0.0)


def grad_bounds(x, w, labels, lse, grad, vocab, ignore, scale, z_weight, dtype, lse_off):
    """(dx bound, dw bound): d is off by its probability's error (the logit's
    and lse's, as factors of the exponential), by the rounding to `dtype`, by the
    probability's own earlier one (an eighth of that, for FP16 a half), and by the
    smallest steps of the 16-bit values (probabilities 2^-32 below a tile's
    largest, d 2^-38 below the largest factor; BF16 2^-64 and none); the sums are fp32
    in any order; results are rounded once."""
    u = HALF_STEP[dtype]
    kept = kept_rows(labels, vocab, ignore)
    dx, dw, d = head_xent_grad(x, w, labels, lse, grad, vocab, ignore, scale, z_weight)
    f = np.abs(scale * grad[kept])
    hit = np.zeros(d.shape)
    hit[np.arange(len(kept)), labels[kept]] = f
    part = np.abs(d + np.where(hit > 0, hit * np.sign(scale * grad[kept])[:, None], 0.0))  # |ca| p
    e = logit_bound(x, w, kept, vocab, scale) + lse_off + 16.0 * U32 * (1 + np.abs(lse[kept]))
    e = e + 4.0 * U32 * scale_mag(x, w, kept, vocab, scale)
    first = 0.5 if dtype == "fp16" else 0.125
    off = part * (1.01 * np.expm1(e)[:, None] + 1.01 * (1 + first) * u + 8 * U32) + hit * (1.01 * u + 8 * U32)
    tiny = 2.0 ** -31 if dtype == "fp16" else 2.0 ** -62
    largest = (f * np.maximum(1.0, np.abs(1 + 2 * z_weight * lse[kept]))).max(initial=0.0)
    off = off + tiny * largest
    big = np.abs(d) + off
    aw, ax = np.abs(w[:vocab]), np.abs(x[kept])
    bx = np.zeros(dx.shape)
    bx[kept] = off @ aw + (2.0 * vocab + 64) * U32 * (big @ aw)
    bw = np.zeros(dw.shape)
    bw[:vocab] = off.T @ ax + (2.0 * len(kept) + 64) * U32 * (big.T @ ax)
    floor = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -130  # results below the smallest normal number
    return bx + u * (np.abs(dx) + bx) + floor, bw, floor
