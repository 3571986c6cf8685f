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


CUT = [(152064, 8192, 26926, 151936), (163840, 7168, 4096, 163840), (163840, 7168, 4096, 32000),
       (163840, 4096, 4096, 128256), (65536, 2048, 8192, 50257), (32768, 1024, 70000, 32000), (163840, 1024, 33, 163840),
       (163840, 7168, 1, 163837), (4096, 264, 33, 4091), (262144, 512, 1 << 20, 262144)]


@pytest.mark.parametrize("kind", [SCORE, GRAD, STEP])
@pytest.mark.parametrize("rows,hidden,m,vocab", CUT)
def test_the_workspace_is_for_the_plan_that_runs(rows, hidden, m, vocab, kind):
    """A call plans for the bytes that it is given: asked again for just that
    many, the plan is the same one. It keeps within the limit unless nothing
    does, and then takes the least."""
    s = shape(rows, hidden, m, vocab)
    whole, least = need(s, kind), need(s, kind, 1)
    limit = whole
    while limit > least // 2:
        n = need(s, kind, limit)
        assert n <= limit or n == least
        assert n >= least
        assert need(s, kind, n) == n
        limit = limit * 7 // 8


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="an accepted call would run on made-up addresses")
@pytest.mark.parametrize("kind", [SCORE, GRAD, STEP])
@pytest.mark.parametrize("rows,hidden,m,vocab", CUT)
def test_less_than_the_least_workspace_is_refused(rows, hidden, m, vocab, kind):
    s = shape(rows, hidden, m, vocab)
    least = need(s, kind, 1)
    lib, p = _lib.lib(), [ctypes.c_void_p(k << 40) for k in range(1, 9)]
    w = _lib.pointer_array([(9 << 40) + r * (rows // 8) * hidden * 2 for r in range(8)])

    def call(nbytes):
        if kind == SCORE:
            return lib.hg_xent(ctypes.byref(s), p[0], w, p[1], p[2], p[3], p[4], nbytes, None)
        if kind == GRAD:
            return lib.hg_xent_grad(ctypes.byref(s), p[0], w, p[1], p[2], p[3], p[4], p[5], 0, 0, p[6], nbytes, None)
        return lib.hg_xent_step(ctypes.byref(s), p[0], w, p[1], p[2], p[3], p[4], p[5], p[6], 0, 0, p[7], nbytes, None)

    assert call(least - 1) == _lib.HG_ESIZE
    assert call(least) != _lib.HG_ESIZE


@pytest.mark.parametrize("rows,hidden,m,vocab", CUT + PADDED)
def test_a_gradient_that_is_not_wanted_takes_no_workspace(rows, hidden, m, vocab):
    s = shape(rows, hidden, m, vocab)
    for limit in (0, GIB):
        both = need(s, GRAD, limit)
        for flag in (_lib.HG_XENT_NO_DX, _lib.HG_XENT_NO_DW):
            n = need(s, GRAD | flag, limit)
            assert need(s, GRAD | flag, n) == n and (limit or n <= both)
    n = ctypes.c_size_t()
    for kind in (GRAD | _lib.HG_XENT_NO_DX | _lib.HG_XENT_NO_DW, STEP | _lib.HG_XENT_NO_DX, SCORE | _lib.HG_XENT_NO_DW,
                 GRAD | 64):
        assert _lib.lib().hg_xent_workspace(ctypes.byref(s), kind, 0, ctypes.byref(n)) == _lib.HG_EINVAL


def test_one_gradient_at_least_is_wanted():
    lib, p, w = _lib.lib(), [ctypes.c_void_p(k << 24) for k in range(1, 9)], _lib.pointer_array([9 << 24])
    s = _lib.XentShape(1, 64, 16, 4, 60, 0, 8, -100, 1.0, 0.0)

    def grad(dx, dw, nbytes=1024):
        return lib.hg_xent_grad(ctypes.byref(s), p[0], w, p[1], p[2], p[3], dx, dw, 0, 0, p[6], nbytes, None)

    assert grad(None, None) == _lib.HG_EINVAL
    assert grad(p[4], None) == grad(None, p[5]) == _lib.HG_ESIZE  # taken, but for the workspace
    assert grad(ctypes.c_void_p((5 << 24) + 8), None) == _lib.HG_EINVAL
