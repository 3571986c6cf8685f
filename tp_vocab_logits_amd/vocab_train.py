"""Training and scoring at the vocabulary matrix: the softmax cross entropy of
the vocab-parallel lm_head product without keeping the logits, the embedding
lookup with scaling, and the gradients of both, through libhg.so.

The matrix is the head weight of :func:`~tp_vocab_logits_amd.head_gather.lmhead`:
``tp`` blocks of ``[shard, hidden]``, block r holding the vocabulary's entries
``r * shard`` and on, given as one ``[tp * shard, hidden]`` (or ``[tp, shard,
hidden]``) tensor or as a sequence of ``tp`` blocks. Gradients come as one
``[tp * shard, hidden]`` tensor; a tied matrix passes the head's gradient to
:func:`embed_grad` as ``dw`` with ``accumulate=True``.

:func:`head_loss` and :func:`embedding` are the differentiable forms for
autograd; the others are the plain calls, whose results carry no history even
if their inputs require gradients. Work is enqueued on the current
stream of the inputs' device; workspaces come from torch's allocator on that
stream. All of it can be captured into a graph.
"""

from __future__ import annotations

import ctypes
import functools
from collections.abc import Iterable

import torch

from . import _lib
from ._lib import check, lib

__all__ = ["head_xent", "head_xent_grad", "head_xent_step", "head_loss", "embed", "embed_grad", "embedding"]

_DTYPES = {torch.bfloat16: _lib.HG_BF16, torch.float16: _lib.HG_FP16, torch.float32: _lib.HG_FP32}

# Workspace a gradient call may take by default: enough for 4096 rows over a
# vocabulary of 163840 in one piece (1.3 GB of 16-bit values, 0.6 GB of partial
# sums), 1.4 % of the card's 288 GB. Larger calls work through the vocabulary
# in pieces.
WORKSPACE_LIMIT = 4 << 30


def _call(fn, name: str, device: torch.device, *args) -> None:
    """One library call on the device's current stream, appended to ``args``."""
    index = device.index
    if torch._C._cuda_getDevice() == index:  # (torch.cuda.current_device() without its check for a first use)
        code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        check(code, name)


def _matrix(w, tp: int, shard: int, dtypes) -> tuple[tuple[int, ...], int, torch.dtype, torch.device]:
    """Block pointers (one for a tensor), hidden size, type and device of the
    vocabulary matrix."""
    tp, shard = int(tp), int(shard)
    if tp < 1 or shard < 1:
        raise ValueError(f"tp and shard must be positive, got {tp} and {shard}")
    if isinstance(w, torch.Tensor):
        if w.dim() not in (2, 3) or not w.is_contiguous() or w.numel() != tp * shard * w.shape[-1]:
            raise ValueError(f"the matrix must be a contiguous [{tp * shard}, H] tensor, got {tuple(w.shape)}")
        if w.dim() == 3 and tuple(w.shape[:2]) != (tp, shard):
            raise ValueError(f"the matrix must be [{tp}, {shard}, H], got {tuple(w.shape)}")
        blocks, hidden = (w,), int(w.shape[-1])
        ptrs = (w.data_ptr(),)
    else:
        if not isinstance(w, Iterable):
            raise ValueError(f"the matrix must be a tensor or {tp} blocks, got {type(w).__name__}")
        blocks = list(w)
        if len(blocks) != tp:
            raise ValueError(f"expected {tp} blocks of the matrix, got {len(blocks)}")
        hidden = int(blocks[0].shape[-1]) if isinstance(blocks[0], torch.Tensor) and blocks[0].dim() else 0
        for t in blocks:
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"every block must be a tensor, got {type(t).__name__}")
            if t.dim() != 2 or tuple(t.shape) != (shard, hidden) or not t.is_contiguous():
                raise ValueError(f"every block must be a contiguous [{shard}, {hidden}] tensor, got {tuple(t.shape)}")
            if t.dtype != blocks[0].dtype or t.device != blocks[0].device:
                raise ValueError("the blocks must share dtype and device")
        ptrs = tuple(t.data_ptr() for t in blocks)
    if blocks[0].dtype not in dtypes:
        raise ValueError(f"the matrix must be one of {[str(d) for d in dtypes]}, got {blocks[0].dtype}")
    return ptrs, hidden, blocks[0].dtype, blocks[0].device


def _given(t, name: str, shape, dtypes, device) -> torch.Tensor:
    """An argument tensor of the given shape, type and device, contiguous."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.is_contiguous() and t.device == device:
        return t
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {' or '.join(str(d) for d in dtypes)} {list(shape)} tensor, "
                         f"got {t.dtype} {list(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the matrix on {device}")
    return t


_INTS = (torch.int64, torch.int32)
_HALVES = (torch.bfloat16, torch.float16)


def _on_gpu(device: torch.device) -> None:
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _xent_bytes(shape: tuple, kind: int, limit: int) -> int:
    """hg_xent_workspace, once per shape: a training loop asks for the same one every step."""
    if limit < 0:  # (a size_t would make it no limit at all)
        raise ValueError(f"workspace_limit must not be negative, got {limit}")
    n = ctypes.c_size_t()
    check(lib().hg_xent_workspace(_lib.XentShape(*shape, 0, 1.0, 0.0), kind, limit, n), "hg_xent_workspace")
    return n.value


_NAMES = {_lib.HG_XENT_SCORE: "hg_xent", _lib.HG_XENT_GRAD: "hg_xent_grad", _lib.HG_XENT_STEP: "hg_xent_step"}


class _Head:
    """The arguments that every cross entropy call shares, checked."""

    def __init__(self, x, w, labels, tp, shard, vocab, ignore, scale, z_weight):
        self.ptrs, hidden, self.dtype, self.device = _matrix(w, tp, shard, _HALVES)
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a [M, H] tensor")
        m = int(x.shape[0])
        self.x = _given(x, "x", (m, hidden), (self.dtype,), self.device)
        self.labels = _given(labels, "labels", (m,), _INTS, self.device)
        _on_gpu(self.device)
        self.m, self.hidden, self.rows = m, hidden, int(tp) * int(shard)
        vocab = self.rows if vocab is None else int(vocab)
        if not 1 <= vocab <= self.rows:
            raise ValueError(f"vocab must lie in 1..{self.rows}, got {vocab}")
        self.shape = (int(tp), int(shard), hidden, m, vocab, _DTYPES[self.dtype], self.labels.element_size())
        self.how = (int(ignore), scale, z_weight)

    def rows_of(self, t, name):
        return _given(t, name, (self.m,), (torch.float32,), self.device)

    def losses(self) -> tuple[torch.Tensor, torch.Tensor]:
        both = torch.empty((2, self.m), dtype=torch.float32, device=self.device)
        return both[0], both[1]

    def grads(self, dx, dw, accumulate):
        if dx is None:
            dx = torch.empty((self.m, self.hidden), dtype=self.dtype, device=self.device)
        else:
            _given(dx, "dx", (self.m, self.hidden), (self.dtype,), self.device)
        return dx, _gradient_buffer(dw, self.rows, self.hidden, self.dtype, self.device, accumulate)

    def call(self, kind, limit, grad, loss, lse, dx, dw, accumulate):
        """The library's call of that kind; addresses of what it does not take are 0."""
        less = 0
        if kind == _lib.HG_XENT_GRAD:
            less = _lib.HG_XENT_NO_DX * (dx is None) | _lib.HG_XENT_NO_DW * (dw is None)
        nbytes = _xent_bytes(self.shape, kind | less, limit)
        ws = _workspace(nbytes, self.device)
        _call(_lib.fast().xent, _NAMES[kind], self.device, kind, self.shape, *self.how, self.x.data_ptr(), self.ptrs,
              self.labels.data_ptr(), grad.data_ptr() if grad is not None else 0,
              loss.data_ptr() if loss is not None else 0, lse.data_ptr(), dx.data_ptr() if dx is not None else 0,
              dw.data_ptr() if dw is not None else 0, int(dw is not None and dw.dtype != self.dtype),
              int(accumulate), ws.data_ptr(), nbytes)


def _gradient_buffer(dw, rows, hidden, dtype, device, accumulate) -> torch.Tensor:
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs the dw to add to")
        return torch.empty((rows, hidden), dtype=dtype, device=device)
    return _given(dw, "dw", (rows, hidden), tuple({dtype, torch.float32}), device)


def head_xent(x: torch.Tensor, w, labels: torch.Tensor, tp: int, shard: int, vocab: int | None = None,
              ignore: int = -100, scale: float = 1.0,
              z_weight: float = 0.0) -> tuple[torch.Tensor, torch.Tensor]:
    """The softmax cross entropy of ``scale * x @ w.T`` per row, and its
    log-sum-exp: ``(loss [M], lse [M])`` in fp32, without keeping the logits.

    ``x`` is ``[M, H]`` BF16 or FP16, ``labels`` ``[M]`` int64 or int32, the
    softmax runs over the first ``vocab`` entries (default: all). ``loss = lse -
    z_label + z_weight * lse**2``; the negated loss at ``z_weight = 0`` is the
    label's log-probability. Rows with the label ``ignore`` get 0 in both; a
    label outside the vocabulary gives NaN. Autograd does not see this call:
    :func:`head_loss` is the differentiable form."""
    h = _Head(x, w, labels, tp, shard, vocab, ignore, scale, z_weight)
    loss, lse = h.losses()
    h.call(_lib.HG_XENT_SCORE, 0, None, loss, lse, None, None, False)
    return loss, lse


def head_xent_grad(x: torch.Tensor, w, labels: torch.Tensor, lse: torch.Tensor, grad: torch.Tensor, tp: int,
                   shard: int, vocab: int | None = None, ignore: int = -100, scale: float = 1.0,
                   z_weight: float = 0.0, dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                   accumulate: bool = False,
                   workspace_limit: int = WORKSPACE_LIMIT) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients ``(dx [M, H], dw [tp*shard, H])`` of ``sum(grad * loss)``
    for the ``lse`` that :func:`head_xent` returned and an upstream ``grad [M]``
    (both fp32). Given, ``dx`` and ``dw`` are written; ``dw`` may be fp32, and
    with ``accumulate`` is added to. The call keeps at most ``workspace_limit``
    bytes of workspace (0: as many as it likes) where the vocabulary can be cut
    into pieces for it."""
    h = _Head(x, w, labels, tp, shard, vocab, ignore, scale, z_weight)
    lse, grad = h.rows_of(lse, "lse"), h.rows_of(grad, "grad")
    dx, dw = h.grads(dx, dw, accumulate)
    h.call(_lib.HG_XENT_GRAD, int(workspace_limit), grad, None, lse, dx, dw, accumulate)
    return dx, dw


def head_xent_step(x: torch.Tensor, w, labels: torch.Tensor, grad: torch.Tensor, tp: int, shard: int,
                   vocab: int | None = None, ignore: int = -100, scale: float = 1.0, z_weight: float = 0.0,
                   dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, accumulate: bool = False,
                   workspace_limit: int = WORKSPACE_LIMIT):
    """Loss and gradients in one call, ``(loss, lse, dx, dw)``, for an upstream
    ``grad [M]`` (fp32) that is known before the loss: the mean's ``1/n``, a
    row's weight. Cheaper than :func:`head_xent` and :func:`head_xent_grad`
    together by one of four products, as the logits are computed once when the
    workspace holds the whole vocabulary."""
    h = _Head(x, w, labels, tp, shard, vocab, ignore, scale, z_weight)
    grad = h.rows_of(grad, "grad")
    loss, lse = h.losses()
    dx, dw = h.grads(dx, dw, accumulate)
    h.call(_lib.HG_XENT_STEP, int(workspace_limit), grad, loss, lse, dx, dw, accumulate)
    return loss, lse, dx, dw


class _HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, labels, tp, shard, how, workspace_limit):
        h = _Head(x, w, labels, tp, shard, **how)
        # two tensors: autograd lets no one change a view that is made in here
        loss, lse = (torch.empty(h.m, dtype=torch.float32, device=h.device) for _ in range(2))
        h.call(_lib.HG_XENT_SCORE, 0, None, loss, lse, None, None, False)
        ctx.save_for_backward(x, w, labels, lse)
        ctx.args = (tp, shard, how, workspace_limit)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, w, labels, lse = ctx.saved_tensors
        tp, shard, how, workspace_limit = ctx.args
        h = _Head(x, w, labels, tp, shard, **how)
        grad = h.rows_of(grad.float().contiguous(), "grad")  # of a sum or mean: one value expanded
        need_x, need_w = ctx.needs_input_grad[:2]
        dx = torch.empty_like(x) if need_x else None
        dw = torch.empty_like(w) if need_w else None
        h.call(_lib.HG_XENT_GRAD, int(workspace_limit), grad, None, lse, dx, dw, False)
        return dx, dw, None, None, None, None, None


def head_loss(x: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, tp: int, shard: int,
              vocab: int | None = None, ignore: int = -100, scale: float = 1.0, z_weight: float = 0.0,
              workspace_limit: int = WORKSPACE_LIMIT) -> torch.Tensor:
    """:func:`head_xent`'s loss ``[M]``, differentiable in ``x`` and ``w`` (one
    tensor). Only ``lse`` is kept for the backward pass, which computes the
    logits again, and the gradients of those that require one, within
    ``workspace_limit`` as :func:`head_xent_grad` does."""
    if not isinstance(w, torch.Tensor):
        raise ValueError("head_loss takes the matrix as one tensor")
    how = {"vocab": vocab, "ignore": ignore, "scale": scale, "z_weight": z_weight}
    return _HeadLoss.apply(x, w, labels, tp, shard, how, workspace_limit)


def _tokens(tokens, device) -> torch.Tensor:
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in _INTS or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int64 or int32 tensor")
    if tokens.device != device:
        raise ValueError(f"tokens are on {tokens.device}, not on {device}")
    return tokens


def embed(tokens: torch.Tensor, w, tp: int, shard: int, scale: float = 1.0,
          out: torch.Tensor | None = None) -> torch.Tensor:
    """Embedding lookup with scaling: ``scale * w[tokens]`` of shape
    ``[*tokens.shape, H]``, rounded once to the matrix's type (BF16, FP16 or
    FP32). A token outside the matrix gives a row of zeros. Autograd does not
    see this call: :func:`embedding` is the differentiable form."""
    ptrs, hidden, dtype, device = _matrix(w, tp, shard, tuple(_DTYPES))
    tokens = _tokens(tokens, device)
    _on_gpu(device)
    shape = (*tokens.shape, hidden)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    else:
        _given(out, "out", shape, (dtype,), device)
    rows = int(tp) * int(shard)  # (blocks that make one tensor are one block)
    _call(_lib.fast().embed, "hg_embed", device, len(ptrs), rows // len(ptrs), hidden, _DTYPES[dtype], ptrs,
          tokens.data_ptr(), tokens.element_size(), tokens.numel(), scale, out.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def _embed_bytes(tp: int, shard: int, hidden: int, n: int) -> int:
    size = ctypes.c_size_t()
    check(lib().hg_embed_workspace(tp, shard, hidden, n, ctypes.byref(size)), "hg_embed_workspace")
    return size.value


def embed_grad(tokens: torch.Tensor, dy: torch.Tensor, tp: int, shard: int, scale: float = 1.0,
               dw: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """The gradient of :func:`embed` in the matrix, ``[tp*shard, H]``: ``dw[v] =
    scale * sum(dy[tokens == v])``, zero where no token names the row. ``dy`` is
    ``[*tokens.shape, H]``. A given ``dw`` (``dy``'s type or fp32) is written,
    or added to with ``accumulate``; sums are fp32 in the order of the tokens."""
    if not isinstance(dy, torch.Tensor) or dy.dtype not in _DTYPES or dy.dim() < 1:
        raise ValueError(f"dy must be one of {[str(d) for d in _DTYPES]}")
    device, hidden = dy.device, int(dy.shape[-1])
    tokens = _tokens(tokens, device)
    _given(dy, "dy", (*tokens.shape, hidden), (dy.dtype,), device)
    _on_gpu(device)
    tp, shard = int(tp), int(shard)
    dw = _gradient_buffer(dw, tp * shard, hidden, dy.dtype, device, accumulate)
    n = tokens.numel()
    nbytes = _embed_bytes(tp, shard, hidden, n)
    ws = _workspace(nbytes, device) if nbytes else None
    _call(_lib.fast().embed_grad, "hg_embed_grad", device, tp, shard, hidden, _DTYPES[dy.dtype], tokens.data_ptr(),
          tokens.element_size(), n, dy.data_ptr(), scale, dw.data_ptr(), int(dw.dtype != dy.dtype), int(accumulate),
          ws.data_ptr() if nbytes else 0, nbytes)
    return dw


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, w, tp, shard, scale):
        ctx.save_for_backward(tokens)
        ctx.args = (tp, shard, scale, w.shape)
        return embed(tokens, w, tp, shard, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        tokens, = ctx.saved_tensors
        tp, shard, scale, shape = ctx.args
        return None, embed_grad(tokens, dy.contiguous(), tp, shard, scale).view(shape), None, None, None


def embedding(tokens: torch.Tensor, w: torch.Tensor, tp: int, shard: int, scale: float = 1.0) -> torch.Tensor:
    """:func:`embed`, differentiable in ``w`` (one tensor)."""
    if not isinstance(w, torch.Tensor):
        raise ValueError("embedding takes the matrix as one tensor")
    return _Embedding.apply(tokens, w, tp, shard, scale)
