"""Low-rank adapters of many requests beside the shared head, through libhg.so:
what each row's adapter adds to the product's shards, and its gradients.

Of ``n`` adapters, adapter i is a pair ``a[i]`` of shape ``[rank, H]`` and
``b[i]`` of shape ``[tp * shard, rank]``, row v for the vocabulary's entry v,
with a factor ``scale[i]``. Row j of a call has adapter ``index[j]``, or none
(-1, or any other value outside ``0 .. n-1``)::

    shards = lmhead(x, w, tp, shard)                                  # [tp, M, shard]
    adapt(shards, x, a, b, index, tp, shard, scale=scale, out=shards)  # in place

:func:`adapted` is the differentiable form for autograd; the others are the
plain calls, whose results carry no history even if their inputs require
gradients. Work is enqueued on the current stream of the inputs' device;
workspaces come from torch's allocator on that stream. All of it can be captured
into a graph.
"""

from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import check, lib
from .vocab_train import _DTYPES, _HALVES, _INTS, _call, _given, _on_gpu, _workspace

__all__ = ["adapt", "adapt_grad", "adapted"]


@functools.lru_cache(maxsize=256)
def _bytes(shape: tuple, kind: int) -> int:
    n = ctypes.c_size_t()
    check(lib().hg_adapt_workspace(_lib.AdaptShape(*shape), kind, n), "hg_adapt_workspace")
    return n.value


class _Adapters:
    """The arguments that every call shares, checked."""

    def __init__(self, y, name, x, a, b, index, tp, shard, scale):
        tp, shard = int(tp), int(shard)
        if tp < 1 or shard < 1:
            raise ValueError(f"tp and shard must be positive, got {tp} and {shard}")
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a [M, H] tensor")
        if not isinstance(a, torch.Tensor) or a.dim() != 3:
            raise ValueError("a must be a [n, rank, H] tensor")
        m, hidden = (int(v) for v in x.shape)
        n, rank = int(a.shape[0]), int(a.shape[1])
        self.device, self.dtype = x.device, x.dtype
        self.x = _given(x, "x", (m, hidden), _HALVES, self.device)
        self.a = _given(a, "a", (n, rank, hidden), (self.dtype,), self.device)
        self.b = _given(b, "b", (n, tp * shard, rank), (self.dtype,), self.device)
        self.index = _given(index, "index", (m,), _INTS, self.device)
        self.scale = None if scale is None else _given(scale, "scale", (n,), (torch.float32,), self.device)
        self.tp, self.columns, self.m = tp, shard, m
        self.y = self.wide(y, name)
        _on_gpu(self.device)
        for what, value, unit in (("shard", shard, 8), ("H", hidden, 8), ("rank", rank, 8)):
            if value < unit or value % unit:
                raise ValueError(f"{what} must be a multiple of {unit}, got {value}")
        if rank > _lib.HG_MAX_RANK or not 1 <= n <= 1 << 15:
            raise ValueError(f"at most {_lib.HG_MAX_RANK} ranks and 1 to {1 << 15} adapters, got {rank} and {n}")
        self.shape = (tp, shard, hidden, m, n, rank, _DTYPES[self.dtype], self.index.element_size())

    def wide(self, t, name):
        """A [tp, M, shard] tensor, or [M, shard] of one block."""
        shape = (self.tp, self.m, self.columns)
        if self.tp == 1 and isinstance(t, torch.Tensor) and t.dim() == 2:
            shape = shape[1:]
        return _given(t, name, shape, (self.dtype,), self.device)

    def call(self, kind, *outputs) -> None:
        nbytes = _bytes(self.shape, kind)
        ws = _workspace(nbytes, self.device)
        fn, name = ((_lib.fast().adapt, "hg_adapt"), (_lib.fast().adapt_grad, "hg_adapt_grad"))[kind]
        _call(fn, name, self.device, self.shape, self.y.data_ptr(), self.x.data_ptr(), self.a.data_ptr(),
              self.b.data_ptr(), self.scale.data_ptr() if self.scale is not None else 0, self.index.data_ptr(),
              *outputs, ws.data_ptr(), nbytes)


def adapt(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor, tp: int,
          shard: int, scale: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """``y`` with what the rows' adapters add: ``y[j] + scale[i] * b[i] @ (a[i] @
    x[j])`` with ``i = index[j]``, rounded once, and ``y[j]`` as it is where a row
    has no adapter.

    ``y`` is the shared product's ``[tp, M, shard]`` (``[M, shard]`` if tp is 1),
    ``x`` its input ``[M, H]``, both BF16 or FP16 as ``a`` and ``b`` are;
    ``index`` is ``[M]`` int64 or int32, ``scale`` ``[n]`` fp32 (default: ones).
    ``out`` may be ``y``: rows without an adapter are then not touched. ``shard``,
    ``H`` and the rank (up to 256) are multiples of 8. :func:`adapted` is the
    differentiable form: autograd does not see this call, only that a given ``out``
    was written, which must not require a gradient while gradients are recorded."""
    if isinstance(out, torch.Tensor) and out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out requires a gradient, which would leave the adapters out: use adapted")
    c = _Adapters(y, "y", x, a, b, index, tp, shard, scale)
    given = out is not None
    if not given:
        out = torch.empty_like(y)
    elif out is not y:
        _given(out, "out", y.shape, (c.dtype,), c.device)
    if c.m:
        c.call(_lib.HG_ADAPT_ADD, out.data_ptr())
        if given:
            increment_version(out)
    return out


def adapt_grad(dy: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor, tp: int,
               shard: int, scale: torch.Tensor | None = None, wide: bool = False,
               need: tuple[bool, bool, bool] = (True, True, True)):
    """The gradients ``(dx [M, H], da [n, rank, H], db [n, tp*shard, rank])`` of
    :func:`adapt` for an upstream ``dy`` of y's shape (which is y's own gradient).

    ``da`` and ``db`` are fp32 if ``wide``, otherwise of the inputs' type, zero
    for an adapter that no row has; ``dx`` is zero for a row without one. ``need``
    says which of the three to compute, the others are None. Sums are fp32 in the
    order of the rows, each result is rounded once. ``n`` times
    rank/64 times the vocabulary/64 (or H/64), rounded up, stays below 2^23."""
    c = _Adapters(dy, "dy", x, a, b, index, tp, shard, scale)
    if len(need) != 3 or not any(need):
        raise ValueError(f"need must name one of dx, da and db at least, got {need}")
    kind = torch.float32 if wide else c.dtype
    dx = torch.empty_like(x) if need[0] else None
    da = torch.empty(a.shape, dtype=kind, device=c.device) if need[1] else None
    db = torch.empty(b.shape, dtype=kind, device=c.device) if need[2] else None
    if c.m or need[1] or need[2]:
        c.call(_lib.HG_ADAPT_GRAD, *(t.data_ptr() if t is not None else 0 for t in (dx, da, db)), int(bool(wide)))
    return dx, da, db


class _Adapted(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, x, a, b, index, tp, shard, scale):
        out = adapt(y, x, a, b, index, tp, shard, scale)
        ctx.save_for_backward(x, a, b, index, scale)
        ctx.args = (tp, shard)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, a, b, index, scale = ctx.saved_tensors
        need = ctx.needs_input_grad[1:4]
        dx = da = db = None
        if any(need):
            dx, da, db = adapt_grad(dy.contiguous(), x, a, b, index, *ctx.args, scale=scale, need=need)
        return dy if ctx.needs_input_grad[0] else None, dx, da, db, None, None, None, None


def adapted(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor, tp: int,
            shard: int, scale: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`adapt` into a new tensor, differentiable in ``y``, ``x``, ``a`` and
    ``b``. Only the inputs are kept for the backward pass, which computes the
    gradients of those that require one; ``scale`` is a constant. As with any
    operator, results that an eager call left must be let go before a backward
    pass of the same leaves is captured: torch cannot capture it otherwise."""
    if scale is not None and scale.requires_grad:
        raise ValueError("adapted has no gradient for scale: it must not require one")
    return _Adapted.apply(y, x, a, b, index, tp, shard, scale)
