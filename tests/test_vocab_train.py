"""The vocabulary matrix's training operators: the oracle against torch's own
cross entropy and embedding in float64 and refusals (CPU); the kernels against
the oracle within bounds derived from their roundings (GPU)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import vocab as ov
from tp_vocab_logits_amd import _lib
from tp_vocab_logits_amd import vocab_train as vt
from tp_vocab_logits_amd._lib import HgError

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu


def note(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def rand(shape, sigma, seed, dtype) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(DT[dtype])


def some_labels(m, vocab, seed, left_out=0.0, ignore=-100) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (m,), generator=g)
    return torch.where(torch.rand(m, generator=g) < left_out, torch.tensor(ignore), t)


# -- the oracle ---------------------------------------------------------------


@pytest.mark.parametrize("scale,z_weight", [(1.0, 0.0), (0.5, 0.0), (1.0, 0.01), (-2.0, 0.1)])
def test_oracle_cross_entropy_is_torchs(scale, z_weight):
    x = torch.randn(7, 12, dtype=torch.float64, requires_grad=True)
    w = torch.randn(20, 12, dtype=torch.float64, requires_grad=True)
    labels = torch.tensor([3, 0, -100, 16, 5, -100, 5])
    g = torch.rand(7, dtype=torch.float64)
    z = scale * (x @ w[:17].t())
    want = torch.nn.functional.cross_entropy(z, labels, reduction="none")
    want = want + z_weight * torch.where(labels == -100, 0.0, torch.logsumexp(z, 1)) ** 2
    (want * g).sum().backward()
    a = (x.detach().numpy(), w.detach().numpy(), labels.numpy())
    loss, lse = ov.head_xent(*a, 17, -100, scale, z_weight)
    np.testing.assert_allclose(loss, want.detach().numpy(), rtol=1e-12)
    dx, dw, _ = ov.head_xent_grad(*a, lse, g.numpy(), 17, -100, scale, z_weight)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-10, atol=1e-14)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-14)


def test_oracle_labels_outside():
    x, w = np.ones((3, 4)), np.ones((6, 4))
    loss, lse = ov.head_xent(x, w, np.array([5, -1, 2]), 5)
    assert np.isnan(loss[:2]).all() and np.isnan(lse[:2]).all() and np.isclose(loss[2], np.log(5))


def test_oracle_embedding_is_torchs():
    w = torch.randn(9, 6, dtype=torch.float64, requires_grad=True)
    tokens = torch.tensor([3, 3, 0, 8, 3])
    out = 2.5 * torch.nn.functional.embedding(tokens, w)
    dy = torch.randn(5, 6, dtype=torch.float64)
    out.backward(dy)
    t = np.array([3, 3, 0, 8, 3])
    np.testing.assert_allclose(ov.embed(t, w.detach().numpy(), 2.5), out.detach().numpy(), rtol=1e-14)
    np.testing.assert_allclose(ov.embed_grad(t, dy.numpy(), 9, 2.5), w.grad.numpy(), rtol=1e-13)
    t = np.array([3, -1, 9, 8, 3])
    assert not ov.embed(t, w.detach().numpy())[[1, 2]].any()
    assert not ov.embed_grad(t, dy.numpy(), 9)[[0, 1, 2, 4, 5, 6, 7]].any()


# -- refusals (no device is touched) -------------------------------------------


def shape(**over):
    s = dict(tp=2, shard=64, hidden=16, m=4, vocab=100, dtype=_lib.HG_BF16, label_bytes=8, ignore=-100, scale=1.0,
             z_weight=0.0)
    s.update(over)
    return _lib.XentShape(**s)


BAD_SHAPES = [dict(tp=0), dict(tp=65), dict(shard=0), dict(shard=48), dict(hidden=0), dict(hidden=12), dict(m=-1),
              dict(vocab=0), dict(vocab=129), dict(dtype=2), dict(dtype=-1), dict(label_bytes=2),
              dict(hidden=(1 << 20) + 8), dict(m=(1 << 24) + 1), dict(m=1 << 24, shard=1 << 20, tp=2),
              dict(hidden=1 << 20, shard=1 << 22, tp=2), dict(hidden=1 << 20, m=1 << 22)]


@pytest.mark.parametrize("over", BAD_SHAPES)
def test_xent_refuses_bad_shapes(over):
    lib, n = _lib.lib(), ctypes.c_size_t()
    s = ctypes.byref(shape(**over))
    w = _lib.pointer_array([1 << 20] * 65)
    p = [ctypes.c_void_p(k << 24) for k in range(1, 9)]
    assert lib.hg_xent_workspace(s, 0, 0, ctypes.byref(n)) == _lib.HG_EINVAL
    assert lib.hg_xent(s, p[0], w, p[1], p[2], p[3], p[4], 1 << 20, None) == _lib.HG_EINVAL
    assert lib.hg_xent_grad(s, p[0], w, p[1], p[2], p[3], p[4], p[5], 0, 0, p[6], 1 << 20, None) == _lib.HG_EINVAL
    assert lib.hg_xent_step(s, p[0], w, p[1], p[2], p[3], p[4], p[5], p[6], 0, 0, p[7], 1 << 20,
                            None) == _lib.HG_EINVAL


def test_xent_workspace_rules():
    lib, n = _lib.lib(), ctypes.c_size_t()

    def need(s, kind, limit=0):
        assert lib.hg_xent_workspace(ctypes.byref(s), kind, limit, ctypes.byref(n)) == _lib.HG_OK
        return n.value

    s = shape()
    assert lib.hg_xent_workspace(ctypes.byref(s), 3, 0, ctypes.byref(n)) == _lib.HG_EINVAL
    assert lib.hg_xent_workspace(ctypes.byref(s), 0, 0, None) == _lib.HG_EINVAL
    assert lib.hg_xent_workspace(None, 0, 0, ctypes.byref(n)) == _lib.HG_EINVAL
    assert need(shape(m=0), 2) == 0
    large = shape(tp=8, shard=20480, hidden=7168, m=4096, vocab=163840)
    for kind in (1, 2):
        whole = need(large, kind)
        assert 2 * 4096 * 163840 < whole < 4 << 30
        for limit in (1 << 30, 768 << 20):
            assert need(large, kind, limit) <= limit, (kind, limit)
        least = need(large, kind, 1)  # the least it can do with
        assert least < whole and need(large, kind, least) <= least
    # d of 2^20 rows: pieces stay within the limit without unbounded search
    assert need(shape(tp=64, shard=4096, hidden=64, m=1 << 20, vocab=1 << 18), 1, 64 << 30) <= 64 << 30


def test_xent_refuses_pointers():
    lib = _lib.lib()
    s = shape()
    size = ctypes.c_size_t()
    assert lib.hg_xent_workspace(ctypes.byref(s), 2, 0, ctypes.byref(size)) == _lib.HG_OK
    base = {"x": 1 << 24, "labels": 2 << 24, "grad": 3 << 24, "loss": 4 << 24, "lse": 5 << 24, "dx": 6 << 24,
            "dw": 7 << 24, "ws": 8 << 24}

    def step(w=(9 << 24, 10 << 24), wide=0, acc=0, nbytes=size.value, **over):
        p = {k: None if v is None else ctypes.c_void_p(v) for k, v in {**base, **over}.items()}
        wp = None if w is None else _lib.pointer_array(w)
        return lib.hg_xent_step(ctypes.byref(s), p["x"], wp, p["labels"], p["grad"], p["loss"], p["lse"], p["dx"],
                                p["dw"], wide, acc, p["ws"], nbytes, None)

    for k in base:
        assert step(**{k: None}) == _lib.HG_EINVAL, k
        assert step(**{k: base[k] + 1}) == _lib.HG_EINVAL, k
    assert step(w=None) == _lib.HG_EINVAL
    assert step(w=(9 << 24, 0)) == _lib.HG_EINVAL
    assert step(w=((9 << 24) + 8, 10 << 24)) == _lib.HG_EINVAL
    assert step(wide=2) == _lib.HG_EINVAL and step(acc=-1) == _lib.HG_EINVAL
    assert step(dx=base["x"]) == _lib.HG_EINVAL          # an output over an input
    assert step(dw=9 << 24) == _lib.HG_EINVAL
    assert step(lse=base["loss"]) == _lib.HG_EINVAL      # two outputs
    assert step(ws=base["dw"]) == _lib.HG_EINVAL
    assert step(nbytes=1024) == _lib.HG_ESIZE
    assert b"workspace" in lib.hg_last_error_detail()


def test_embed_refusals():
    lib = _lib.lib()
    n = ctypes.c_size_t()
    w = _lib.pointer_array([1 << 24, 2 << 24])
    tok, out, ws = (ctypes.c_void_p(k << 24) for k in (3, 4, 5))

    def look(tp=2, shard=64, hidden=16, dtype=0, w=w, tok=tok, tb=8, k=4, out=out):
        return lib.hg_embed(tp, shard, hidden, dtype, w, tok, tb, k, 1.0, out, None)

    def grad(tp=2, shard=64, hidden=16, dtype=0, tok=tok, tb=8, k=4, dy=ctypes.c_void_p(1 << 24), dw=out, wide=0,
             acc=0, ws=ws, nbytes=1 << 20):
        return lib.hg_embed_grad(tp, shard, hidden, dtype, tok, tb, k, dy, 1.0, dw, wide, acc, ws, nbytes, None)

    for f in (look, grad):
        for bad in (dict(tp=0), dict(tp=65), dict(shard=0), dict(hidden=4), dict(hidden=0), dict(dtype=3),
                    dict(tb=2), dict(k=-1), dict(tok=None), dict(tok=ctypes.c_void_p((3 << 24) + 4))):
            assert f(**bad) == _lib.HG_EINVAL, (f, bad)
    assert look(w=None) == _lib.HG_EINVAL and look(out=None) == _lib.HG_EINVAL
    assert look(out=ctypes.c_void_p(1 << 24)) == _lib.HG_EINVAL
    assert look(k=0) == _lib.HG_OK  # nothing to do
    assert grad(dw=None) == _lib.HG_EINVAL and grad(dy=None) == _lib.HG_EINVAL
    assert grad(k=300, ws=None) == _lib.HG_EINVAL and grad(k=300, ws=ctypes.c_void_p((5 << 24) + 64)) == _lib.HG_EINVAL
    assert grad(dw=ctypes.c_void_p(1 << 24)) == _lib.HG_EINVAL and grad(wide=2) == _lib.HG_EINVAL
    assert grad(k=300, nbytes=64) == _lib.HG_ESIZE
    assert grad(k=0, acc=1) == _lib.HG_OK
    assert lib.hg_embed_workspace(2, 64, 16, 4, None) == _lib.HG_EINVAL
    assert lib.hg_embed_workspace(2, 64, 16, -1, ctypes.byref(n)) == _lib.HG_EINVAL
    assert lib.hg_embed_workspace(2, 64, 16, 0, ctypes.byref(n)) == _lib.HG_OK and n.value == 0
    assert lib.hg_embed_workspace(2, 64, 16, 300, ctypes.byref(n)) == _lib.HG_OK and n.value > 0


def test_python_refusals():
    x, w, t = torch.zeros(3, 16, dtype=torch.bfloat16), torch.zeros(64, 16, dtype=torch.bfloat16), torch.zeros(3).long()
    g = torch.zeros(3)
    for bad in (dict(x=x.float()), dict(x=x[:, :8]), dict(x=x[0]), dict(w=w.float()), dict(w=w[:32]), dict(w=[w, w]),
                dict(w=w.t().contiguous().t()), dict(labels=g), dict(labels=t[:2]), dict()):
        a = {"x": x, "w": w, "labels": t, **bad}  # the last one: not on a GPU
        with pytest.raises(ValueError):
            vt.head_xent(a["x"], a["w"], a["labels"], 1, 64)
    with pytest.raises(ValueError):
        vt.head_xent(x, w, t, 0, 64)
    for bad in (t.float(), torch.zeros(4, 2).long().t()):
        with pytest.raises(ValueError):
            vt.embed(bad, w, 1, 64)
    with pytest.raises(ValueError):
        vt.embed(t, w, 1, 64)  # not on a GPU
    with pytest.raises(ValueError):
        vt.embed_grad(t, x[:2], 1, 64)
    with pytest.raises(ValueError):
        vt.embed_grad(t, x, 1, 64)
    with pytest.raises(ValueError):
        vt.head_loss(x, [w], t, 1, 64)
    with pytest.raises(ValueError):
        vt.embedding(t, [w], 1, 64)


# -- the cross entropy on the GPU -----------------------------------------------


class Problem:
    def __init__(self, tp, shard, hidden, m, vocab=None, dtype="bf16", left_out=0.0, scale=1.0, z_weight=0.0, seed=0,
                 sigma=0.2, blocks=False, ints=torch.int64):
        self.tp, self.shard, self.vocab, self.dtype = tp, shard, vocab or tp * shard, dtype
        self.x = rand((m, hidden), 1.0, 100 + seed, dtype)
        self.w = rand((tp * shard, hidden), sigma, 200 + seed, dtype)
        self.labels = some_labels(m, self.vocab, 300 + seed, left_out).to(ints)
        self.grad = torch.rand(m, generator=torch.Generator().manual_seed(400 + seed)) / m
        self.how = {"vocab": self.vocab, "ignore": -100, "scale": scale, "z_weight": z_weight}
        self.blocks = blocks

    def on_gpu(self):
        w = self.w.to(DEV)
        if self.blocks:  # blocks that do not follow one another in memory
            room = torch.full((self.tp, self.shard + 1, w.shape[1]), float("nan"), dtype=w.dtype, device=DEV)
            room[:, :self.shard] = w.view(self.tp, self.shard, -1)
            w = [room[r, :self.shard] for r in range(self.tp)]
        return self.x.to(DEV), w, self.labels.to(DEV), self.grad.to(DEV)

    def wanted(self, lse=None):
        a = (f64(self.x), f64(self.w), self.labels.long().numpy())
        loss, exact = ov.head_xent(*a, **self.how)
        return a, loss, exact

    def check_loss(self, loss, lse):
        a, want, exact = self.wanted()
        kept = ov.kept_rows(a[2], self.vocab, -100)
        loss, lse = f64(loss), f64(lse)
        rest = np.setdiff1d(np.arange(len(want)), kept)
        assert np.array_equal(loss[rest], want[rest], equal_nan=True)
        assert np.array_equal(lse[rest], exact[rest], equal_nan=True)
        how = self.how
        b = ov.lse_bound(a[0], a[1], kept, self.vocab, how["scale"], exact)
        assert (np.abs(lse[kept] - exact[kept]) <= b).all(), np.abs(lse[kept] - exact[kept]).max()
        b = ov.loss_bound(a[0], a[1], kept, self.vocab, how["scale"], how["z_weight"], exact)
        assert (np.abs(loss[kept] - want[kept]) <= b).all(), np.abs(loss[kept] - want[kept]).max()

    def check_grads(self, dx, dw, lse_used=None, old=None):
        """lse_used: the lse that the call was given (float64); its error is
        then none of the call's."""
        a, _, exact = self.wanted()
        kept = ov.kept_rows(a[2], self.vocab, -100)
        lse = exact if lse_used is None else lse_used
        off = (ov.lse_bound(a[0], a[1], kept, self.vocab, self.how["scale"], exact) if lse_used is None
               else np.zeros(len(kept)))
        g = f64(self.grad)
        how = self.how
        want_x, want_w, _ = ov.head_xent_grad(*a, lse, g, **how)
        bx, bw, floor = ov.grad_bounds(*a, lse, g, self.vocab, -100, how["scale"], how["z_weight"], self.dtype, off)
        assert dx.dtype == self.x.dtype
        bad = np.abs(f64(dx) - want_x) > bx
        assert not bad.any(), (int(bad.sum()), np.abs(f64(dx) - want_x).max())
        if old is not None:
            want_w = want_w + old
        wide = dw.dtype == torch.float32
        u, floor = (ov.U32, 2.0 ** -140) if wide else (ov.HALF_STEP[self.dtype], floor)
        bw = bw + u * (np.abs(want_w) + bw) + floor + (4 * ov.U32 * np.abs(old) if old is not None else 0)
        bad = np.abs(f64(dw) - want_w) > bw
        assert not bad.any(), (int(bad.sum()), np.abs(f64(dw) - want_w).max())


SIZES = [  # tp, shard, hidden, m, vocab
    (1, 32, 8, 1, None), (1, 32, 8, 1, 1), (2, 32, 72, 3, 33), (2, 64, 64, 17, 127), (3, 288, 136, 33, 800),
    (8, 96, 512, 256, None), (4, 160, 264, 257, 639), (64, 32, 64, 5, 2047), (2, 1024, 40, 300, 1000),
    (1, 2272, 200, 64, 2245), (5, 160, 64, 1000, 513), (2, 512, 1032, 511, None)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,vocab", SIZES)
def test_loss_against_oracle(tp, shard, hidden, m, vocab, dtype):
    note(f"head_xent {tp=} {shard=} {hidden=} {m=} {vocab=} {dtype}")
    p = Problem(tp, shard, hidden, m, vocab, dtype, left_out=0.2 if m > 4 else 0.0)
    x, w, t, _ = p.on_gpu()
    loss, lse = vt.head_xent(x, w, t, tp, shard, **p.how)
    p.check_loss(loss, lse)
    again = vt.head_xent(x, w, t, tp, shard, **p.how)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,vocab", SIZES)
def test_step_against_oracle(tp, shard, hidden, m, vocab, dtype):
    note(f"head_xent_step {tp=} {shard=} {hidden=} {m=} {vocab=} {dtype}")
    p = Problem(tp, shard, hidden, m, vocab, dtype, left_out=0.2 if m > 4 else 0.0, scale=0.7, z_weight=0.01)
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, tp, shard, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)
    again = vt.head_xent_step(x, w, t, g, tp, shard, **p.how)
    for a, b in zip((loss, lse, dx, dw), again):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,vocab", SIZES)
def test_grad_against_oracle(tp, shard, hidden, m, vocab, dtype):
    note(f"head_xent_grad {tp=} {shard=} {hidden=} {m=} {vocab=} {dtype}")
    p = Problem(tp, shard, hidden, m, vocab, dtype, left_out=0.2 if m > 4 else 0.0, scale=-0.5, z_weight=0.02, seed=1)
    x, w, t, g = p.on_gpu()
    lse = torch.from_numpy(p.wanted()[2]).float()
    dx, dw = vt.head_xent_grad(x, w, t, lse.to(DEV), g, tp, shard, **p.how)
    p.check_grads(dx, dw, lse_used=f64(lse))


@gpu
@pytest.mark.parametrize("tp,shard,hidden,m", [(3, 96, 200, 70), (2, 512, 64, 300), (9, 32, 72, 5)])
def test_blocks_apart_in_memory(tp, shard, hidden, m):
    note(f"blocks apart {tp=} {shard=} {hidden=} {m=}")
    p = Problem(tp, shard, hidden, m, tp * shard - 5, "bf16", 0.1)
    x, w, t, g = p.on_gpu()
    together = vt.head_xent_step(x, w, t, g, tp, shard, **p.how)
    p.blocks = True
    _, apart, _, _ = p.on_gpu()
    for a, b in zip(together, vt.head_xent_step(x, apart, t, g, tp, shard, **p.how)):
        assert torch.equal(a, b)
    p.check_grads(*together[2:])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("m", [1, 130])
def test_accumulating_and_wide_gradients(dtype, wide, m):
    note(f"accumulate {dtype} {wide=} {m=}")
    p = Problem(2, 320, 136, m, 601, dtype, 0.1)
    x, w, t, g = p.on_gpu()
    old = rand((640, 136), 1e-2, 5, "fp32" if wide else dtype).to(DEV)
    dw = old.clone()
    _, _, dx, out = vt.head_xent_step(x, w, t, g, 2, 320, dw=dw, accumulate=True, **p.how)
    assert out is dw
    p.check_grads(dx, dw, old=f64(old))
    assert torch.equal(dw[601:], old[601:])  # rows past the vocabulary keep their values
    if wide:
        _, _, dx, dw = vt.head_xent_step(x, w, t, g, 2, 320, dw=torch.full_like(old, float("nan")), **p.how)
        p.check_grads(dx, dw)


@gpu
@pytest.mark.parametrize("tp,shard,hidden,m,vocab", [(4, 512, 136, 300, 2001), (3, 288, 64, 33, 800)])
def test_vocabulary_in_pieces(tp, shard, hidden, m, vocab):
    note(f"pieces {tp=} {shard=} {hidden=} {m=} {vocab=}")
    p = Problem(tp, shard, hidden, m, vocab, "bf16", 0.2, z_weight=0.01)
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, tp, shard, workspace_limit=1, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)
    dx, dw = vt.head_xent_grad(x, w, t, lse, g, tp, shard, workspace_limit=1, **p.how)
    p.check_grads(dx, dw, lse_used=f64(lse))


@gpu
@pytest.mark.parametrize("split", [(64, 32, 64, 3000, 2047), (1, 256, 1024, 2500, 250)])
def test_long_sums_are_split(split):
    """Few tiles and a long sum: both products run split."""
    tp, shard, hidden, m, vocab = split
    note(f"split {split}")
    p = Problem(tp, shard, hidden, m, vocab, "bf16", 0.5, sigma=0.05)
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, tp, shard, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)


@gpu
@pytest.mark.parametrize("m", [0, 1, 40])
def test_no_row_counts(m):
    note(f"no row counts {m=}")
    p = Problem(2, 96, 64, m, 150)
    x, w, _, g = p.on_gpu()
    t = torch.full((m,), -100, device=DEV)
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 2, 96, dw=torch.full((192, 64), 7.0, device=DEV).bfloat16(),
                                          **p.how)
    assert loss.shape == lse.shape == (m,) and dx.shape == (m, 64)
    assert not loss.any() and not lse.any() and not dx.any() and not dw.any()
    assert [v.numel() for v in vt.head_xent(x, w, t, 2, 96, **p.how)] == [m, m]
    dx, dw = vt.head_xent_grad(x, w, t, lse, g, 2, 96, **p.how)
    assert not dx.any() and not dw.any()
    old = dw + 3
    vt.head_xent_grad(x, w, t, lse, g, 2, 96, dw=old, accumulate=True, **p.how)
    assert (old == 3).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_masked_places_hold_anything(dtype, bad):
    """Rows left out and matrix rows past the vocabulary: whatever they hold
    reaches no result."""
    note(f"masked places {dtype} {bad}")
    p = Problem(2, 160, 72, 40, 301, dtype, 0.3)
    x, w, t, g = p.on_gpu()
    clean = vt.head_xent_step(x, w, t, g, 2, 160, **p.how)
    v = torch.finfo(DT[dtype]).min if bad == "lowest" else bad
    x[t == -100] = v
    w[301:] = v
    g[t == -100] = float("nan")
    for a, b in zip(clean, vt.head_xent_step(x, w, t, g, 2, 160, **p.how)):
        assert torch.equal(a, b)
    lse = clean[1].masked_fill(t == -100, float("nan"))
    dx, dw = vt.head_xent_grad(x, w, t, lse, g, 2, 160, **p.how)
    p.check_grads(dx, dw, lse_used=f64(clean[1]))
    loss, lse = vt.head_xent(x, w, t, 2, 160, **p.how)
    p.check_loss(loss, lse)


@gpu
def test_labels_outside_the_vocabulary():
    note("labels outside")
    p = Problem(2, 96, 64, 9, 150)
    p.labels[[1, 4, 7]] = torch.tensor([150, -1, 2 ** 40])
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 2, 96, **p.how)
    assert torch.isnan(loss[[1, 4, 7]]).all() and torch.isnan(lse[[1, 4, 7]]).all()
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)


@gpu
def test_int32_labels_and_another_ignored_value():
    note("int32 labels")
    p = Problem(2, 96, 64, 30, 150, left_out=0.3, ints=torch.int32)
    x, w, t, g = p.on_gpu()
    a = vt.head_xent_step(x, w, t, g, 2, 96, **p.how)
    p.check_loss(*a[:2])
    t = torch.where(t == -100, 5, torch.where(t == 5, 6, t)).long()
    b = vt.head_xent_step(x, w, t, g, 2, 96, **{**p.how, "ignore": 5})
    keep = p.labels.to(DEV) != 5
    for u, v in zip(a[:3], b[:3]):
        assert torch.equal(u[keep], v[keep])


@gpu
def test_confident_rows():
    """Logits far apart: a probability of one beside others that vanish."""
    note("confident rows")
    p = Problem(1, 512, 64, 20, dtype="fp16", sigma=1.0, seed=3)
    p.x = p.x * 4
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 1, 512, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)
    # every label the row's largest logit
    p.labels = torch.from_numpy(np.argmax(f64(p.x) @ f64(p.w).T, axis=1))
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 1, 512, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)


@gpu
@pytest.mark.parametrize("factor", [0.0, 1e-30, 1e30, -1.0])
def test_upstream_gradients_of_any_size(factor):
    note(f"upstream {factor}")
    p = Problem(2, 96, 64, 30, 150, dtype="bf16")
    p.grad = p.grad * factor
    x, w, t, g = p.on_gpu()
    _, _, dx, dw = vt.head_xent_step(x, w, t, g, 2, 96, **p.how)
    p.check_grads(dx, dw)


@gpu
def test_gradient_against_differences():
    """x and its neighbours are exact in BF16: x on a grid of 1/16, steps of
    1/64, |x| < 2. The central difference of one row's loss is off by h^2/6 of
    the third derivative (at most the third power of the span of a column of W)
    and by the loss's own bound over h."""
    note("differences")
    p = Problem(2, 96, 64, 12, 150)
    p.x = (torch.round(p.x.float().clamp(-1.9, 1.9) * 16) / 16).bfloat16()
    p.grad = torch.ones(12)
    x, w, t, g = p.on_gpu()
    dx, _ = vt.head_xent_step(x, w, t, g, 2, 96, **p.how)[2:]
    h = 1 / 64
    a, _, exact = p.wanted()
    noise = ov.loss_bound(a[0], a[1], np.arange(12), 150, 1.0, 0.0, exact) * 1.5
    for k in (0, 17, 63):
        up, down = x.clone(), x.clone()
        up[:, k] += h
        down[:, k] -= h
        diff = (f64(vt.head_xent(up, w, t, 2, 96, **p.how)[0]) - f64(vt.head_xent(down, w, t, 2, 96, **p.how)[0])) / (2 * h)
        span = np.ptp(a[1][:150, k])
        bound = h * h / 6 * span ** 3 + noise / h + ov.HALF_STEP["bf16"] * 4 * span
        assert (np.abs(f64(dx)[:, k] - diff) <= bound).all()


@gpu
def test_autograd_and_torchs_formula():
    note("autograd")
    p = Problem(2, 96, 64, 50, 150, left_out=0.2)
    x, w, t, _ = p.on_gpu()
    x.requires_grad_(), w.requires_grad_()
    n = int((p.labels != -100).sum())
    loss = vt.head_loss(x, w, t, 2, 96, **p.how)
    (loss.sum() / n).backward()
    p.grad = torch.full((50,), 1 / n)
    lse = vt.head_xent(x.detach(), w.detach(), t, 2, 96, **p.how)[1]
    p.check_grads(x.grad, w.grad, lse_used=f64(lse))
    # twice: gradients add up
    vt.head_loss(x, w, t, 2, 96, **p.how).mean().backward()
    assert x.grad.isfinite().all()


@gpu
def test_graph_replays_and_another_stream():
    note("graph")
    p = Problem(2, 320, 136, 70, 601, left_out=0.1)
    x, w, t, g = p.on_gpu()
    tokens = torch.randint(-1, 640, (90,), generator=torch.Generator().manual_seed(1)).to(DEV)
    dy = rand((90, 136), 1.0, 2, "bf16").to(DEV)

    def both():
        loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 2, 320, **p.how)
        vt.embed_grad(tokens, dy, 2, 320, dw=dw, accumulate=True)
        return loss, lse, dx, dw, vt.embed(tokens, w, 2, 320, 3.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in range(4):
        x.copy_(rand(x.shape, 1.0, 50 + k, "bf16"))
        t.copy_(some_labels(70, 601, 60 + k, 0.1 * k))
        want = [v.clone() for v in both()]
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


# -- the embedding on the GPU ----------------------------------------------------


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tp,shard,hidden,n", [(1, 1, 8, 1), (2, 33, 16, 7), (3, 5, 2056, 40), (8, 96, 7168, 5),
                                               (64, 2, 72, 300)])
@pytest.mark.parametrize("scale", [1.0, 11.313708])
def test_lookup(tp, shard, hidden, n, dtype, scale):
    note(f"embed {tp=} {shard=} {hidden=} {n=} {dtype} {scale}")
    w = rand((tp * shard, hidden), 1.0, 7, dtype)
    tokens = torch.randint(-2, tp * shard + 2, (n,), generator=torch.Generator().manual_seed(n))
    want = ov.embed(tokens.numpy(), f64(w), float(np.float32(scale)))
    for ints in (torch.int64, torch.int32):
        got = vt.embed(tokens.to(ints).to(DEV), w.to(DEV), tp, shard, scale)
        assert got.dtype == w.dtype and got.shape == (n, hidden)
        # one fp32 product, one rounding
        bound = (ov.HALF_STEP[dtype] + 2 * ov.U32) * np.abs(want) + 2.0 ** -25 * (dtype == "fp16")
        assert (np.abs(f64(got) - want) <= bound).all()
    if scale == 1.0:
        inside = (tokens >= 0) & (tokens < tp * shard)
        assert torch.equal(got.cpu()[inside], w[tokens[inside]])  # values unchanged
    blocks = [w.view(tp, shard, hidden)[r].clone().to(DEV) for r in range(tp)]
    assert torch.equal(vt.embed(tokens.to(DEV), blocks, tp, shard, scale), got)


def check_embed_grad(tokens, dy, tp, shard, scale, dtype, wide=False, old=None):
    rows = tp * shard
    count = np.bincount(tokens[(tokens >= 0) & (tokens < rows)].numpy(), minlength=rows)
    want = ov.embed_grad(tokens.numpy(), f64(dy), rows, float(np.float32(scale)))
    mag = np.abs(ov.embed_grad(tokens.numpy(), np.abs(f64(dy)), rows, float(np.float32(scale))))
    dw = None
    if wide or old is not None:
        dw = torch.full((rows, dy.shape[-1]), float("nan"), device=DEV, dtype=torch.float32 if wide else dy.dtype)
        if old is not None:
            dw.copy_(old)
            want = want + f64(old)
            mag = mag + np.abs(f64(old))
    got = vt.embed_grad(tokens.to(DEV), dy.to(DEV), tp, shard, scale, dw=dw, accumulate=old is not None)
    u = ov.U32 if wide else ov.HALF_STEP[dtype]
    off = (count[:, None] + 4) * 1.01 * ov.U32 * mag
    bound = off + u * (np.abs(want) + off) + 2.0 ** -25 * (dtype == "fp16" and not wide)
    bad = np.abs(f64(got) - want) > bound
    assert not bad.any(), (int(bad.sum()), np.abs(f64(got) - want).max())
    if old is None:
        assert not got[torch.from_numpy(count == 0)].any()
    else:
        untouched = torch.from_numpy(count == 0)
        assert torch.equal(got.cpu()[untouched], old[untouched].to(got.dtype))
    return got


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tp,shard,hidden,n", [(1, 1, 8, 1), (2, 33, 16, 7), (1, 513, 72, 64), (3, 5, 2056, 400), (2, 40, 2056, 256),
                                               (2, 40, 72, 257),
                                               (8, 96, 264, 4096), (8, 96, 264, 4097), (64, 300, 40, 9000),
                                               (5, 70000, 8, 5000), (64, 5000, 264, 9001)])
def test_embed_grad(tp, shard, hidden, n, dtype):
    note(f"embed_grad {tp=} {shard=} {hidden=} {n=} {dtype}")
    rows = tp * shard
    g = torch.Generator().manual_seed(n)
    rank = torch.exp(torch.rand(n, generator=g) * np.log(rows + 1)).long() - 1  # frequent tokens among them
    tokens = torch.where(torch.rand(n, generator=g) < 0.1, -1, (rank * 7919) % rows)
    dy = rand((n, hidden), 1.0, 11, dtype)
    a = check_embed_grad(tokens, dy, tp, shard, 2.0, dtype)
    b = vt.embed_grad(tokens.to(torch.int32).to(DEV), dy.to(DEV), tp, shard, 2.0)
    assert torch.equal(a, b)  # the same bits, whatever the integers' width
    old = rand((rows, hidden), 1.0, 12, dtype)
    check_embed_grad(tokens, dy, tp, shard, 0.5, dtype, old=old)
    if dtype != "fp32":
        check_embed_grad(tokens, dy, tp, shard, 2.0, dtype, wide=True)
        check_embed_grad(tokens, dy, tp, shard, 2.0, dtype, wide=True, old=old.float())


@gpu
@pytest.mark.parametrize("n", [1, 63, 64, 65, 256, 257, 1000, 4096, 20000])
def test_embed_grad_of_one_token(n):
    """Every position the same token: one sum through every block."""
    note(f"one token {n=}")
    dy = rand((n, 40), 1.0, 13, "bf16")
    check_embed_grad(torch.full((n,), 17), dy, 2, 30, 1.0, "bf16")


@gpu
@pytest.mark.parametrize("n", [0, 5, 5000])
def test_embed_grad_without_tokens(n):
    note(f"no tokens {n=}")
    dy = torch.full((n, 40), float("nan")).bfloat16()
    tokens = torch.where(torch.arange(n) % 2 == 0, -1, 60)
    check_embed_grad(tokens, dy, 2, 30, 1.0, "bf16")
    check_embed_grad(tokens, dy, 2, 30, 1.0, "bf16", old=rand((60, 40), 1.0, 3, "bf16"))


@gpu
def test_embedding_autograd_in_two_dimensions():
    note("embedding autograd")
    w = rand((96, 64), 1.0, 1, "bf16").to(DEV).requires_grad_()
    tokens = torch.randint(0, 96, (4, 9), generator=torch.Generator().manual_seed(3))
    out = vt.embedding(tokens.to(DEV), w, 2, 48, 8.0)
    assert out.shape == (4, 9, 64)
    dy = rand((4, 9, 64), 1.0, 4, "bf16")
    out.backward(dy.to(DEV))
    want = ov.embed_grad(tokens.view(-1).numpy(), f64(dy).reshape(36, 64), 96, 8.0)
    mag = ov.embed_grad(tokens.view(-1).numpy(), np.abs(f64(dy)).reshape(36, 64), 96, 8.0)
    off = 40 * ov.U32 * mag
    assert (np.abs(f64(w.grad) - want) <= off + ov.HALF_STEP["bf16"] * (np.abs(want) + off)).all()


@gpu
def test_argument_rules_on_device():
    x, w = rand((3, 64), 1.0, 1, "bf16").to(DEV), rand((96, 64), 1.0, 2, "bf16").to(DEV)
    t, g = torch.zeros(3, dtype=torch.long, device=DEV), torch.zeros(3, device=DEV)
    with pytest.raises(ValueError):
        vt.head_xent(x, w, t.cpu(), 2, 48)  # labels elsewhere
    with pytest.raises(HgError):
        vt.head_xent(x, w, t, 2, 48)        # shard % 32
    with pytest.raises(ValueError):
        vt.head_xent(x, w, t, 1, 96, vocab=97)
    with pytest.raises(ValueError):
        vt.head_xent_step(x, w, t, g.double(), 1, 96)
    with pytest.raises(ValueError):
        vt.head_xent_step(x, w, t, g, 1, 96, accumulate=True)  # nothing to add to
    with pytest.raises(HgError):
        vt.head_xent_step(x, w, t, g, 1, 96, dw=w)             # over an input
    with pytest.raises(ValueError):
        vt.embed(t, w, 1, 95)
    with pytest.raises(ValueError):
        vt.embed_grad(t, x.double(), 1, 96)


@gpu
@pytest.mark.parametrize("m", [1, 15, 16, 17, 31, 32, 33, 64, 65, 100, 127, 128, 129])
@pytest.mark.parametrize("tp,shard,hidden,vocab", [(1, 32, 8, 5), (8, 2592, 136, 20700), (1, 12320, 328, 12301),
                                                   (2, 20512, 72, 41001)])
def test_few_rows(tp, shard, hidden, vocab, m):
    """Up to 128 rows the matrix is streamed, by row counts rounded up to 16,
    32, 64 and 128; the vocabulary's runs end inside tiles and units."""
    note(f"few rows {tp=} {shard=} {hidden=} {vocab=} {m=}")
    p = Problem(tp, shard, hidden, m, vocab, "bf16", 0.1, scale=1.5, z_weight=0.01)
    x, w, t, _ = p.on_gpu()
    x = torch.cat([x, torch.full_like(x, float("nan"))])[:m]  # rows past m hold anything
    w[vocab:] = float("nan")
    loss, lse = vt.head_xent(x, w, t, tp, shard, **p.how)
    p.check_loss(loss, lse)
    p.blocks = True
    again = vt.head_xent(x, p.on_gpu()[1], t, tp, shard, **p.how)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@gpu
def test_the_example_learns():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "tied_vocab_training.py")
    spec = importlib.util.spec_from_file_location("tied_vocab_training", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    note("example")
    losses = example.train(40, tell=note)
    assert np.isfinite(losses).all()
    assert abs(losses[0] - np.log(1000)) < 1.0 and losses[-1] < 0.8 * losses[0]
    assert losses == example.train(40, tell=note)  # the same bits every time


@gpu
@pytest.mark.parametrize("m", [8, 200])
def test_losses_of_certain_rows_keep_their_digits(m):
    """Labels far above the other logits: losses down to 1e-6, from logits
    around 20. The logits here are exact (a product of few powers of two), so
    the loss may be off by the exponentials and sums alone: a handful of fp32
    roundings of numbers about 1 and of the loss itself."""
    note(f"certain rows {m=}")
    vocab, hidden = 640, 64
    x = torch.zeros(m, hidden)
    x[:, 0] = 1.0
    x[:, 1] = torch.arange(m) % 8 * 0.25
    w = torch.zeros(vocab, hidden)
    w[:, 0] = torch.randint(0, 9, (vocab,), generator=torch.Generator().manual_seed(1)) * 0.25
    w[7, 0], w[7, 1] = 19.0, 1.0
    labels = torch.full((m,), 7)
    loss, lse = vt.head_xent(x.bfloat16().to(DEV), w.bfloat16().to(DEV), labels.to(DEV), 2, 320)
    want, exact = ov.head_xent(x.numpy().astype(float), w.numpy().astype(float), labels.numpy(), vocab)
    assert (np.abs(f64(loss) - want) <= 64 * ov.U32 * want + 4 * ov.U32).all()
    assert (np.abs(f64(lse) - exact) <= 16 * ov.U32 * exact).all()
    g = torch.full((m,), 1.0 / m)
    step = vt.head_xent_step(x.bfloat16().to(DEV), w.bfloat16().to(DEV), labels.to(DEV), g.to(DEV), 2, 320)
    assert (np.abs(f64(step[0]) - want) <= 64 * ov.U32 * want + 4 * ov.U32).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,vocab", [(2, 8480, 520, 300, 16901), (1, 17408, 264, 513, 17001),
                                                     (3, 5696, 776, 129, None), (2, 8480, 72, 1100, 16640)])
def test_big_tiles(tp, shard, hidden, m, vocab, dtype):
    """Sizes whose 256 x 256 tiles occupy more than half of the CUs (in the
    logits, the gradients or both), with edges inside tiles, rows left out and
    a matrix that ends tiles past the vocabulary."""
    note(f"big tiles {tp=} {shard=} {hidden=} {m=} {vocab=} {dtype}")
    p = Problem(tp, shard, hidden, m, vocab, dtype, left_out=0.15, scale=0.8, z_weight=0.01, sigma=0.1)
    x, w, t, g = p.on_gpu()
    out = vt.head_xent_step(x, w, t, g, tp, shard, **p.how)
    p.check_loss(*out[:2])
    p.check_grads(*out[2:])
    lse = torch.from_numpy(p.wanted()[2]).float()
    dx, dw = vt.head_xent_grad(x, w, t, lse.to(DEV), g, tp, shard, **p.how)
    p.check_grads(dx, dw, lse_used=f64(lse))
    old = rand((tp * shard, hidden), 1e-2, 5, "fp32").to(DEV)
    wide = old.clone()
    vt.head_xent_step(x, w, t, g, tp, shard, dw=wide, accumulate=True, **p.how)
    p.check_grads(out[2], wide, old=f64(old))
    # blocks apart in memory, and anything in the masked places: the same bits
    p.blocks = tp > 1
    _, w, _, _ = p.on_gpu()
    x[t == -100] = float("nan")
    g[t == -100] = float("inf")
    if tp == 1:
        w[p.vocab:] = float("nan")
    elif p.vocab < tp * shard:
        w[-1][p.vocab - (tp - 1) * shard:] = float("nan")
    for a, b in zip(out, vt.head_xent_step(x, w, t, g, tp, shard, **p.how)):
        assert torch.equal(a, b)
    # the vocabulary in pieces
    limit = vt._xent_bytes(vt._Head(x, w, t, tp, shard, **p.how).shape, _lib.HG_XENT_STEP, 0) * 2 // 3
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, tp, shard, workspace_limit=limit, **p.how)
    assert torch.equal(loss, out[0]) and torch.equal(lse, out[1])
    p.check_grads(dx, dw)


def test_fastcall_wrappers_pass_arguments_on():
    """The fast-call wrappers of the training operators reach the entry points:
    bad shapes give their codes, malformed calls raise before reaching C."""
    f = _lib.fast()
    dims = (2, 64, 16, 4, 100, 0, 8)
    rest = (1 << 24, (9 << 24,), 2 << 24, 3 << 24, 4 << 24, 5 << 24, 6 << 24, 7 << 24, 0, 0, 8 << 24, 1 << 10, 0)
    for kind in (0, 1, 2):
        assert f.xent(kind, (2, 48, 16, 4, 96, 0, 8), -100, 1.0, 0.0, *rest) == _lib.HG_EINVAL  # shard % 32
        assert f.xent(kind, dims, -100, 1.0, 0.0, *rest) == _lib.HG_ESIZE                       # 1 KB of workspace
    assert f.xent(3, dims, -100, 1.0, 0.0, *rest) == _lib.HG_EINVAL
    assert f.xent(0, (65, 64, 16, 4, 100, 0, 8), -100, 1.0, 0.0, *rest) == _lib.HG_EINVAL
    with pytest.raises(TypeError):
        f.xent(0, dims[:6], -100, 1.0, 0.0, *rest)
    with pytest.raises(TypeError):
        f.xent(0, dims, -100, 1.0, 0.0, 1 << 24, (1, 2, 3), *rest[2:])
    with pytest.raises(TypeError):
        f.xent(0, dims, -100, "1", 0.0, *rest)
    assert f.embed(1, 64, 16, 3, (1 << 24,), 2 << 24, 8, 4, 1.0, 3 << 24, 0) == _lib.HG_EINVAL
    with pytest.raises(TypeError):
        f.embed(2, 64, 16, 0, (1 << 24,), 2 << 24, 8, 4, 1.0, 3 << 24, 0)
    assert f.embed_grad(1, 64, 16, 0, 1 << 24, 8, 4, 2 << 24, 1.0, 0, 0, 0, 0, 0, 0) == _lib.HG_EINVAL
    assert f.embed_grad(1, 64, 16, 0, 0, 8, 0, 0, 1.0, 16, 0, 1, 0, 0, 0) == _lib.HG_OK  # nothing to add
