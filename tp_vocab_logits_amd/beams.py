"""Beam search on the logits, through libhg.so: which continuations of each
request's beams to keep, and the beams' states (token histories, caches) put
in their order.

A request has ``beams`` rows, row ``q * beams + k`` is beam k of request q: in
the logits, in the scores and in every state. A step of a search that keeps
``beams`` of them::

    scores, parents, tokens = beam_select(logits, scores, beams)
    beam_reorder(caches, parents, lengths, time_dim=2)      # in place

Work is enqueued on the current stream of the inputs' device; the workspace
comes from torch's allocator on that stream. Both can be captured into a
graph. Autograd sees neither, but for the version of the states, so that a
backward pass notices if it needs one that was reordered; states that require a
gradient are refused.
"""

from __future__ import annotations

import ctypes
import functools
import math
from collections.abc import Iterable

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import check, lib
from .vocab_train import _DTYPES, _INTS, _call, _given, _on_gpu, _workspace

__all__ = ["beam_select", "beam_reorder"]


@functools.lru_cache(maxsize=256)
def _select_bytes(requests, beams, keep, tp, shard, vocab, dtype) -> int:
    n = ctypes.c_size_t()
    check(lib().hg_beam_workspace(_lib.BeamShape(requests, beams, keep, tp, shard, vocab, dtype, 0, 1.0), n),
          "hg_beam_workspace")
    return n.value


def _logits(logits, rows: int) -> tuple[tuple[int, ...], int, torch.dtype, torch.device]:
    """Block pointers, row width, type and device of the logits."""
    if isinstance(logits, torch.Tensor):
        shape = tuple(logits.shape)
        if len(shape) not in (2, 3) or not logits.is_contiguous():
            raise ValueError("logits must be a contiguous [rows, vocab] or [tp, rows, shard] tensor, or blocks, got "
                             f"{list(shape)}{'' if logits.is_contiguous() else ', not contiguous'}")
        tp = shape[0] if len(shape) == 3 else 1
        if not 1 <= tp <= _lib.HG_MAX_TP or shape[-2] != rows or shape[-1] < 1:
            raise ValueError(f"logits must have {rows} rows (one per beam of each request) in 1 to {_lib.HG_MAX_TP} "
                             f"blocks, got {list(shape)}")
        if logits.dtype not in _DTYPES:
            raise ValueError(f"logits must be one of {[str(d) for d in _DTYPES]}, got {logits.dtype}")
        at, step = logits.data_ptr(), rows * shape[-1] * logits.element_size()
        return tuple(range(at, at + tp * step, step)) if rows else (at,) * tp, shape[-1], logits.dtype, logits.device
    if not isinstance(logits, Iterable):
        raise ValueError(f"logits must be a tensor or blocks, got {type(logits).__name__}")
    blocks = list(logits)
    if not 1 <= len(blocks) <= _lib.HG_MAX_TP:
        raise ValueError(f"the logits must have 1 to {_lib.HG_MAX_TP} blocks, got {len(blocks)}")
    first = blocks[0]
    for t in blocks:
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_contiguous():
            raise ValueError("every block of the logits must be a contiguous [rows, shard] tensor")
        if t.shape != first.shape or t.dtype != first.dtype or t.device != first.device:
            raise ValueError("the blocks must share shape, dtype and device")
    if first.dtype not in _DTYPES:
        raise ValueError(f"logits must be one of {[str(d) for d in _DTYPES]}, got {first.dtype}")
    if first.shape[0] != rows or first.shape[1] < 1:
        raise ValueError(f"logits must have {rows} rows (one per beam of each request), got {list(first.shape)}")
    return tuple(t.data_ptr() for t in blocks), int(first.shape[1]), first.dtype, first.device


def beam_select(logits, scores: torch.Tensor, keep: int, vocab: int | None = None, scale: float = 1.0,
                finished: torch.Tensor | None = None,
                pad: int = 0) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The ``keep`` best continuations of each request, ``(scores, parents,
    tokens)``, each ``[requests, keep]`` in descending order: over the request's
    beams k and the tokens v, ``scores[k] + log_softmax(scale * logits[k])[v]``.

    ``logits`` are gathered rows ``[requests * beams, vocab]`` or the product's
    shards ``[tp, requests * beams, shard]`` (or tp blocks), BF16, FP16 or FP32;
    the softmax runs over the first ``vocab`` entries (default: all), ``scale`` is
    taken as fp32. ``scores``
    is ``[requests, beams]`` fp32, minus infinity (or any other value that is not
    finite) for a beam that is not there, such as all but one at the start. Equal
    candidates go by beam, then token; sums and order are in 64 bits, of
    exponentials to 1e-10.

    Tokens whose logit is minus infinity or NaN are no candidates. With
    ``finished`` (``[requests, beams]`` bool), a finished beam stands for itself:
    its score unchanged, token ``pad``. ``parents`` is the beam (int64), -1 as
    the token and a score of minus infinity where candidates run out. ``keep``
    and the beams go to 64."""
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores must be a [requests, beams] tensor")
    requests, beams = (int(v) for v in scores.shape)
    ptrs, shard, dtype, device = _logits(logits, requests * beams)
    _given(scores, "scores", (requests, beams), (torch.float32,), device)
    if finished is not None:
        _given(finished, "finished", (requests, beams), (torch.bool,), device)
    _on_gpu(device)
    keep, pad, tp = int(keep), int(pad), len(ptrs)
    vocab = tp * shard if vocab is None else int(vocab)
    if not 1 <= beams <= _lib.HG_MAX_BEAMS or not 1 <= keep <= _lib.HG_MAX_KEEP:
        raise ValueError(f"beams and keep must lie in 1..{_lib.HG_MAX_BEAMS}, got {beams} and {keep}")
    if not 1 <= vocab <= min(tp * shard, 1 << 20):
        raise ValueError(f"vocab must lie in 1..{min(tp * shard, 1 << 20)}, got {vocab}")
    if not 0 <= pad < vocab:
        raise ValueError(f"pad must lie in 0..{vocab - 1}, got {pad}")
    if not 0.0 < scale < math.inf:
        raise ValueError(f"scale must be positive and finite, got {scale}")
    out = torch.empty((requests, keep), dtype=torch.float32, device=device)
    parents, tokens = (torch.empty((requests, keep), dtype=torch.int64, device=device) for _ in range(2))
    if requests:
        nbytes = _select_bytes(requests, beams, keep, tp, shard, vocab, _DTYPES[dtype])
        ws = _workspace(nbytes, device)
        _call(_lib.fast().beam_select, "hg_beam_select", device,
              (requests, beams, keep, shard, vocab, _DTYPES[dtype], pad), scale, ptrs, scores.data_ptr(),
              finished.data_ptr() if finished is not None else 0, out.data_ptr(), parents.data_ptr(),
              tokens.data_ptr(), ws.data_ptr(), nbytes)
    return out, parents, tokens


def _merged(sizes, strides) -> list[list[int]]:
    """The dimensions, outermost first, with those that continue each other as
    one; dimensions of one entry are dropped."""
    out: list[list[int]] = []
    for n, step in zip(sizes, strides):
        if n == 1:
            continue
        if out and out[-1][1] == n * step:
            out[-1] = [out[-1][0] * n, step]
        else:
            out.append([n, step])
    return out


@functools.lru_cache(maxsize=1024)
def _geometry(shape, strides, size: int, time_dim: int | None) -> tuple[int, int, int, int, int]:
    """``(row_stride, outer_stride, step_bytes, outer, steps)`` of a state."""
    if not shape:
        raise ValueError("a state must have a dimension of beams")
    if 0 in shape:
        return 0, 0, 0, 0, 0
    steps, split = 1, len(shape)
    if time_dim is not None:
        if not 1 <= time_dim < len(shape):
            raise ValueError(f"time_dim must name a dimension after the beams', got {time_dim} for {list(shape)}")
        steps, split = shape[time_dim], time_dim
    where = f"a state of shape {list(shape)} and strides {list(strides)}"
    inner = _merged(shape[split:], strides[split:])  # the run: positions and what follows
    outer = _merged(shape[1:split], strides[1:split])
    if time_dim is None and outer and outer[-1][1] == 1:
        inner = [outer.pop()]
    if len(inner) > 1 or (inner and inner[0][1] != 1):
        raise ValueError(f"{where} must be without gaps from {'its positions' if time_dim is not None else 'its end'} on")
    if len(outer) > 1:
        raise ValueError(f"{where} has more than one run of rows in strides: pass parts of it")
    run = inner[0][0] if inner else 1
    many, step = outer[0] if outer else (1, 0)
    return strides[0] * size, step * size, run // steps * size, many, steps


def beam_reorder(states, parents: torch.Tensor, lengths: torch.Tensor | None = None,
                 time_dim: int | None = None) -> None:
    """Puts the beams' states in the order of ``parents``, in place: row ``q *
    beams + k`` of each state becomes what row ``q * beams + parents[q, k]`` was.

    ``states`` is a tensor or a sequence of them, of any types, each with
    ``requests * beams`` rows in its first dimension. ``parents`` is ``[requests,
    beams]`` int64 or int32, as :func:`beam_select` returns it; a parent outside
    the beams (-1) leaves its row as it is. With ``lengths`` (``[requests]``,
    int64 or int32) only the first ``lengths[q]`` positions along ``time_dim``
    move (clamped to what there is), the others keep their values. A state must
    be without gaps from ``time_dim`` on; states must not overlap (views of one
    cache may lie between each other's rows)."""
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise ValueError("parents must be a [requests, beams] tensor")
    requests, beams = (int(v) for v in parents.shape)
    device = parents.device
    _given(parents, "parents", (requests, beams), _INTS, device)
    if not 1 <= beams <= _lib.HG_MAX_BEAMS:
        raise ValueError(f"beams must lie in 1..{_lib.HG_MAX_BEAMS}, got {beams}")
    if lengths is not None:
        _given(lengths, "lengths", (requests,), _INTS, device)
        if time_dim is None:
            raise ValueError("lengths need the time_dim that they count")
    states = (states,) if isinstance(states, torch.Tensor) else tuple(states)
    table = []
    for t in states:
        if not isinstance(t, torch.Tensor) or t.device != device or t.layout != torch.strided:
            raise ValueError(f"every state must be a tensor on {device}")
        if t.dim() < 1 or t.shape[0] != requests * beams:
            raise ValueError(f"every state must have {requests * beams} rows, got {list(t.shape)}")
        if t.requires_grad:
            raise ValueError("a state that requires a gradient cannot be reordered in place")
        dim = time_dim + t.dim() if time_dim is not None and time_dim < 0 else time_dim
        table.append((t.data_ptr(), _geometry(tuple(t.shape), t.stride(), t.element_size(), dim)))
    _on_gpu(device)
    if requests and table:
        _call(_lib.fast().beam_reorder, "hg_beam_reorder", device, requests, beams, tuple(table), parents.data_ptr(),
              parents.element_size(), lengths.data_ptr() if lengths is not None else 0,
              lengths.element_size() if lengths is not None else 0)
        increment_version(states)
