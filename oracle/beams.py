"""Oracle of the beam search operators: plain float64 definitions, one row and
one request at a time. Test infrastructure only; shares nothing with the
library."""

from __future__ import annotations

import numpy as np


def log_probabilities(z: np.ndarray) -> np.ndarray:
    """Log-softmax of one row in float64: NaN counts as minus infinity, the
    infinite ones of a row share its probability, a row of nothing is minus
    infinity throughout."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64))
    top = z.max()
    if top == -np.inf:
        return np.full_like(z, -np.inf)
    if top == np.inf:
        return np.where(z == np.inf, -np.log(np.count_nonzero(z == np.inf)), -np.inf)
    return z - (top + np.log(np.exp(z - top).sum()))


def candidates(logits, scores, finished=None, pad=0, scale=1.0) -> np.ndarray:
    """``[requests, beams, vocab]``: every candidate's score, minus infinity
    where there is none. ``logits`` is ``[requests, beams, vocab]``."""
    logits, scores = np.asarray(logits, dtype=np.float64), np.asarray(scores, dtype=np.float64)
    out = np.full(logits.shape, -np.inf)
    for q, k in np.ndindex(*scores.shape):
        if not np.isfinite(scores[q, k]):
            continue
        if finished is not None and finished[q, k]:
            out[q, k, pad] = scores[q, k]
        else:
            out[q, k] = scores[q, k] + log_probabilities(float(scale) * logits[q, k])
    return out


def beam_select(logits, scores, keep, finished=None, pad=0, scale=1.0):
    """``(scores, parents, tokens)``, each ``[requests, keep]``."""
    c = candidates(logits, scores, finished, pad, scale)
    requests, _, vocab = c.shape
    out = np.full((requests, keep), -np.inf)
    parents = np.full((requests, keep), -1, dtype=np.int64)
    tokens = parents.copy()
    for q in range(requests):
        flat = c[q].reshape(-1)
        order = np.lexsort((np.arange(flat.size), -flat))[:keep]
        order = order[flat[order] > -np.inf]
        out[q, : order.size] = flat[order]
        parents[q, : order.size], tokens[q, : order.size] = np.divmod(order, vocab)
    return out, parents, tokens


def beam_reorder(state, parents, lengths=None, time_dim=None) -> np.ndarray:
    """The reordered copy of one state (rows in its first dimension)."""
    state, new = np.asarray(state), np.array(state)
    beams = parents.shape[1]
    for (q, k), p in np.ndenumerate(parents):
        if not 0 <= p < beams:
            continue
        part = [slice(None)] * (state.ndim - 1)
        if lengths is not None:
            part[time_dim - 1] = slice(0, max(0, int(lengths[q])))
        new[(q * beams + k, *part)] = state[(q * beams + int(p), *part)]
    return new
