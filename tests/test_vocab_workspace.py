"""The cross entropy's workspace: what hg_xent_workspace asks for, against what
it is asked to keep within (CPU); gradients of a matrix that goes on long past
its vocabulary (GPU)."""

from __future__ import annotations

import ctypes

import pytest
import torch

from tp_vocab_logits_amd import _lib
from tp_vocab_logits_amd import vocab_train as vt

DEV = "cuda:0"
SCORE, GRAD, STEP = _lib.HG_XENT_SCORE, _lib.HG_XENT_GRAD, _lib.HG_XENT_STEP
GIB = 1 << 30


def shape(rows, hidden, m, vocab, tp=8, dtype=_lib.HG_BF16):
    return _lib.XentShape(tp, rows // tp, hidden, m, vocab, dtype, 8, -100, 1.0, 0.0)


def need(s, kind, limit=0) -> int:
    n = ctypes.c_size_t()
    assert _lib.lib().hg_xent_workspace(ctypes.byref(s), kind, limit, ctypes.byref(n)) == _lib.HG_OK
    return n.value


# matrix rows, hidden, m, vocabulary: from none to most of the matrix past the vocabulary
PADDED = [(163840, 1024, 4096, 50257), (163840, 7168, 4096, 32000), (163840, 4096, 4096, 128256),
          (163840, 2048, 4096, 256), (163840, 2048, 4096, 1), (1 << 20, 1024, 4096, 256), (65536, 264, 33, 4091),
          (32768, 4096, 777, 32767)]


@pytest.mark.parametrize("kind", [GRAD, STEP])
@pytest.mark.parametrize("rows,hidden,m,vocab", PADDED)
def test_rows_past_the_vocabulary_take_no_workspace(rows, hidden, m, vocab, kind):
    """The same bytes as for a matrix that ends with its vocabulary."""
    ends = -(-vocab // 256) * 256
    for limit in (0, GIB, 64 << 20):
        assert need(shape(rows, hidden, m, vocab), kind, limit) == need(shape(ends, hidden, m, vocab), kind, limit)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,hidden,m,vocab", [(16384, 136, 3000, 250), (16384, 136, 3000, 257), (2048, 520, 40, 1),
                                                 (20480, 1032, 300, 16900)])
def test_gradients_end_with_the_vocabulary(rows, hidden, m, vocab, dtype):
    """With and without partial sums, on both tiles: rows past the vocabulary
    become zeros, or keep every bit when accumulating."""
    print(f"[gpu] past the vocabulary {rows=} {hidden=} {m=} {vocab=} {dtype}", flush=True)
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.randn(m, hidden, generator=g, device=DEV).to(t)
    w = (torch.randn(rows, hidden, generator=g, device=DEV) * 0.1).to(t)
    w[vocab:] = float("nan")
    labels = torch.randint(0, vocab, (m,), generator=g, device=DEV)
    grad = torch.rand(m, generator=g, device=DEV)
    ends = -(-vocab // 256) * 256
    short = vt.head_xent_step(x, w[:ends], labels, grad, 1, ends, vocab=vocab)
    for wide in (False, True):
        old = torch.full((rows, hidden), float("nan"), dtype=torch.float32 if wide else t, device=DEV)
        got = vt.head_xent_step(x, w, labels, grad, 8, rows // 8, vocab=vocab, dw=old.clone())
        for a, b in zip(got[:3], short[:3]):
            assert torch.equal(a, b)
        assert not got[3][vocab:].any()
        if not wide:
            assert torch.equal(got[3][:ends], short[3])
        old[:vocab] = 0.25
        old[vocab::2] = -0.0
        dw = old.clone()
        vt.head_xent_step(x, w, labels, grad, 8, rows // 8, vocab=vocab, dw=dw, accumulate=True)
        bits = torch.int32 if wide else torch.int16
        assert torch.equal(dw[vocab:].view(bits), old[vocab:].view(bits))
        assert dw[:vocab].isfinite().all()
