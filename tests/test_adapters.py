"""Low-rank adapters of many requests: the oracle against torch in float64 and
against differences, argument checks and refusals (CPU); the kernels against the
oracle within bounds derived from their roundings (GPU)."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import adapters as oa
from tp_vocab_logits_amd import _lib, adapt, adapt_grad, adapted
from tp_vocab_logits_amd._lib import HgError

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu


def note(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs on the CPU, in the call's types."""

    def __init__(self, dtype, tp, shard, hidden, m, n, rank, *, run=1, left_out=0.2, scaled=True, seed=0, sigma=1.0,
                 index=torch.int64):
        g = torch.Generator().manual_seed(seed + 1000 * m + rank)
        t = DT[dtype]
        self.kind, self.tp, self.shard = dtype, tp, shard
        many = -(-m // run)
        who = torch.randint(0, n, (many,), generator=g)
        out = torch.rand(many, generator=g) < left_out
        who = torch.where(out, torch.where(torch.rand(many, generator=g) < 0.5, -1, n + 3), who)
        self.index = who.repeat_interleave(run)[:m].contiguous().to(index)
        self.x = torch.randn(m, hidden, generator=g).to(t)
        self.a = (torch.randn(n, rank, hidden, generator=g) / math.sqrt(hidden)).to(t)
        self.b = (torch.randn(n, tp * shard, rank, generator=g) * 0.1).to(t)
        self.scale = torch.rand(n, generator=g) + 0.5 if scaled else None
        self.y = (torch.randn(tp, m, shard, generator=g) * sigma).to(t)

    def flat(self, y):
        """[tp, M, shard] -> [M, V]"""
        return f64(y.transpose(0, 1).reshape(y.shape[1], -1)) if y.shape[1] else np.zeros((0, self.tp * self.shard))

    def low(self):
        return (f64(self.x), f64(self.a), f64(self.b), self.index.numpy(),
                None if self.scale is None else f64(self.scale))

    def on(self, device):
        return [t.to(device) for t in (self.x, self.a, self.b, self.index)]

    def how(self, device):
        return dict(scale=None if self.scale is None else self.scale.to(device))

    def check(self, got, y=None):
        want, bound = oa.adapt_bound(self.flat(self.y if y is None else y), *self.low(), self.kind)
        got = self.flat(got)
        assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / (bound + 1e-300))
        # in the norm: every element's own rounding, and what the bounds' typical parts come to
        norm = np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= norm * (oa.HALF_STEP[self.kind] + 2.0 ** -14) + 1e-6

    def check_grads(self, got, dy, wide=False, need=(True, True, True)):
        out = "fp32" if wide else self.kind
        wants, bounds = oa.adapt_grad_bound(self.flat(dy), *self.low(), self.kind, out)
        for name, t, want, bound, kind, asked in zip("dx da db".split(), got, wants, bounds, (self.kind, out, out), need):
            if not asked:
                assert t is None
                continue
            assert t.dtype == DT[kind], name
            e = np.abs(f64(t) - want)
            assert (e <= bound).all(), (name, np.max(e / (bound + 1e-300)))
            assert np.linalg.norm(e) <= np.linalg.norm(want) * (oa.HALF_STEP[kind] + 2.0 ** -14) + 1e-6, name


# -- the oracle ---------------------------------------------------------------


def small():
    return Case("fp32", 2, 8, 24, 11, 3, 8, seed=4)


def test_oracle_is_torchs_and_its_gradient_autograds():
    c = small()
    x, a, b, _, s = (torch.from_numpy(v).requires_grad_(v.dtype == np.float64) for v in c.low())
    y = torch.from_numpy(c.flat(c.y)).requires_grad_()
    live = torch.nonzero((c.index >= 0) & (c.index < 3)).squeeze(1)
    i = c.index[live].long()
    more = torch.einsum("mrh,mh->mr", a[i], x[live])
    out = y.index_add(0, live, s[i][:, None] * torch.einsum("mvr,mr->mv", b[i], more))
    np.testing.assert_allclose(oa.adapt(y.detach().numpy(), *c.low()), out.detach().numpy(), rtol=1e-12, atol=1e-14)
    dy = torch.randn(out.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(5))
    out.backward(dy)
    for got, want in zip(oa.adapt_grad(dy.numpy(), *c.low()), (x, a, b)):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_oracle_gradient_is_the_differences():
    c = small()
    y, low = c.flat(c.y), list(c.low())
    dy = np.random.RandomState(3).randn(*y.shape)
    grads = oa.adapt_grad(dy, *low)
    rng = np.random.RandomState(4)
    for k in range(3):  # (linear in each alone)
        step = rng.randn(*low[k].shape)
        ends = []
        for sign in (1, -1):
            moved = list(low)
            moved[k] = low[k] + sign * 1e-3 * step
            ends.append((oa.adapt(y, *moved) * dy).sum())
        np.testing.assert_allclose((ends[0] - ends[1]) / 2e-3, (grads[k] * step).sum(), rtol=1e-9)


# -- refusals -----------------------------------------------------------------


def test_arguments_are_checked():
    c = Case("bf16", 2, 8, 16, 5, 3, 8)
    good = dict(y=c.y, x=c.x, a=c.a, b=c.b, index=c.index, tp=2, shard=8, scale=c.scale)
    for bad in (dict(y=c.y[:, :4]), dict(y=c.y.half()), dict(y=c.y.transpose(0, 1)), dict(x=c.x[0]), dict(x=None),
                dict(x=c.x.float()), dict(a=c.a[0]), dict(a=c.a[:, :, :8]), dict(b=c.b[:2]), dict(b=c.b.half()),
                dict(b=c.b.transpose(1, 2)), dict(index=c.index[:4]), dict(index=c.index.float()),
                dict(index=c.index.to(torch.int16)), dict(scale=c.scale.double()), dict(scale=c.scale[:2]),
                dict(tp=0), dict(shard=0), dict(tp=1), dict(shard=4)):
        with pytest.raises(ValueError):
            adapt(**{**good, **bad})
        if "y" not in bad:
            args = {**good, **bad}
            args["dy"] = args.pop("y")
            with pytest.raises(ValueError):
                adapt_grad(**args)
    with pytest.raises(ValueError, match="CUDA"):
        adapt(**good)
    with pytest.raises(ValueError, match="scale"):
        adapted(**{**good, "scale": c.scale.requires_grad_()})


def shape(**more):
    return _lib.AdaptShape(**{**dict(tp=2, shard=16, hidden=24, m=5, adapters=3, rank=8, dtype=_lib.HG_BF16,
                                     index_bytes=8), **more})


def test_library_checks_shapes():
    lib = _lib.lib()
    n = ctypes.c_size_t()
    for kind in (_lib.HG_ADAPT_ADD, _lib.HG_ADAPT_GRAD):
        assert lib.hg_adapt_workspace(shape(), kind, n) == 0 and n.value > 0
        assert lib.hg_adapt_workspace(shape(m=0), kind, n) == 0 and n.value == 0
        for bad in (dict(tp=0), dict(tp=65), dict(shard=0), dict(shard=12), dict(hidden=0), dict(hidden=20),
                    dict(hidden=(1 << 20) + 8), dict(m=-1), dict(m=(1 << 24) + 1), dict(adapters=0),
                    dict(adapters=(1 << 15) + 1), dict(rank=0), dict(rank=12), dict(rank=264), dict(dtype=_lib.HG_FP32),
                    dict(index_bytes=2), dict(tp=64, shard=1 << 23), dict(m=1 << 24, shard=1 << 16)):
            assert lib.hg_adapt_workspace(shape(**bad), kind, n) == _lib.HG_EINVAL, bad
        assert lib.hg_adapt_workspace(None, kind, n) == lib.hg_adapt_workspace(shape(), kind, None) == _lib.HG_EINVAL
    assert lib.hg_adapt_workspace(shape(), 2, n) == _lib.HG_EINVAL
    # more strips of gradients than a launch covers
    assert lib.hg_adapt_workspace(shape(adapters=1 << 15, shard=1 << 15), _lib.HG_ADAPT_GRAD, n) == _lib.HG_EINVAL


def test_library_checks_pointers():
    lib = _lib.lib()
    mb = 1 << 20
    y, x, a, b, s, i, out, ws = (k * mb for k in range(1, 9))

    def call(fn=lib.hg_adapt, at=None, value=None, size=mb, sh=None, more=()):
        args = [y, x, a, b, s, i, out, *more, ws]
        if at is not None:
            args[at] = value
        return fn(sh or shape(), *args, size, None)

    assert call(size=16) == _lib.HG_ESIZE
    for at in (0, 1, 2, 3, 5, 6, 7):
        assert call(at=at, value=None) == _lib.HG_EINVAL, at
    for at in (0, 1, 2, 3, 6, 7):
        assert call(at=at, value=(at + 1) * mb + 8) == _lib.HG_EINVAL, at
    assert call(at=4, value=s + 2) == call(at=5, value=i + 4) == _lib.HG_EINVAL
    for other in (x, a, b, s, i):
        assert call(at=6, value=other) == call(at=7, value=other) == _lib.HG_EINVAL  # overlaps
    assert call(at=6, value=y + 16) == _lib.HG_EINVAL  # into y, not y itself
    assert call(sh=shape(m=0), at=0, value=None) == _lib.HG_OK
    grad = lib.hg_adapt_grad
    more = (9 * mb, 10 * mb, 0)  # da, db, wide
    assert call(grad, more=more, size=16) == _lib.HG_ESIZE
    assert call(grad, more=(9 * mb, 10 * mb, 2)) == _lib.HG_EINVAL
    assert call(grad, at=6, value=None, more=(None, None, 0)) == _lib.HG_EINVAL
    assert call(grad, more=(9 * mb + 8, 10 * mb, 0)) == call(grad, more=(9 * mb, 10 * mb + 4, 0)) == _lib.HG_EINVAL
    assert call(grad, more=(9 * mb, 9 * mb + 16, 0)) == call(grad, more=(a, 10 * mb, 0)) == _lib.HG_EINVAL
    assert call(grad, at=6, value=y, more=more) == _lib.HG_EINVAL
    assert call(grad, sh=shape(m=0), at=6, value=None, more=(None, None, 0)) == _lib.HG_EINVAL


# -- on the GPU ---------------------------------------------------------------

SHAPES = [  # tp, shard, hidden, m, n, rank, rows per request
    (1, 8, 8, 1, 1, 8, 1), (8, 20480, 7168, 1, 8, 16, 1), (2, 2056, 264, 1, 2, 64, 1), (1, 72, 40, 15, 3, 16, 1),
    (2, 64, 512, 16, 1, 8, 16), (3, 136, 520, 17, 20, 24, 1), (4, 200, 1032, 33, 3, 32, 4), (2, 1000, 264, 63, 63, 8, 1),
    (8, 256, 768, 64, 32, 16, 1), (2, 2048, 264, 65, 7, 40, 2), (1, 4096, 1024, 130, 4, 64, 33),
    (3, 328, 776, 200, 40, 72, 1), (2, 120, 96, 257, 5, 128, 50), (1, 264, 200, 100, 2, 256, 10),
    (2, 72, 72, 1000, 300, 16, 1), (1, 1032, 136, 4099, 6, 8, 700)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,n,rank,run", SHAPES)
def test_adapters(dtype, tp, shard, hidden, m, n, rank, run):
    note(f"adapt {dtype} {tp} {shard} {hidden} {m} {n} {rank} {run}")
    c = Case(dtype, tp, shard, hidden, m, n, rank, run=run)
    got = adapt(c.y.to(DEV), *c.on(DEV), tp, shard, **c.how(DEV))
    c.check(got)
    bare = torch.nonzero((c.index < 0) | (c.index >= n)).squeeze(1)
    assert torch.equal(got.cpu()[:, bare], c.y[:, bare])
    place = c.y.to(DEV)
    assert adapt(place, *c.on(DEV), tp, shard, out=place, **c.how(DEV)) is place
    assert torch.equal(place, got)


@gpu
@pytest.mark.parametrize("dtype,wide", [("bf16", False), ("bf16", True), ("fp16", False), ("fp16", True)])
@pytest.mark.parametrize("tp,shard,hidden,m,n,rank,run", SHAPES)
def test_gradients(dtype, wide, tp, shard, hidden, m, n, rank, run):
    if shard == 20480:
        n = 2  # (the oracle's time)
    note(f"adapt grad {dtype} {wide} {tp} {shard} {hidden} {m} {n} {rank} {run}")
    c = Case(dtype, tp, shard, hidden, m, n, rank, run=run, seed=1, sigma=0.01)
    got = adapt_grad(c.y.to(DEV), *c.on(DEV), tp, shard, wide=wide, **c.how(DEV))
    c.check_grads(got, c.y, wide)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m,n,rank,run", [
    (2, 328, 264, 300, 2, 40, 60), (1, 264, 72, 200, 1, 64, 200), (3, 520, 136, 513, 3, 24, 17), (2, 64, 520, 129, 2, 16, 9),
    (4, 1000, 1032, 1100, 5, 64, 1), (1, 8, 8, 65, 1, 8, 65), (2, 2048, 264, 4100, 8, 48, 333)])
def test_many_rows_of_few_adapters(dtype, tp, shard, hidden, m, n, rank, run):
    """The second product that keeps its columns and goes through the rows."""
    note(f"adapt stream {dtype} {tp} {shard} {hidden} {m} {n} {rank} {run}")
    assert m > 64 and m // 64 >= n and rank <= 64
    c = Case(dtype, tp, shard, hidden, m, n, rank, run=run, seed=2, sigma=0.5)
    got = adapt(c.y.to(DEV), *c.on(DEV), tp, shard, **c.how(DEV))
    c.check(got)
    place = c.y.to(DEV)
    adapt(place, *c.on(DEV), tp, shard, out=place, **c.how(DEV))
    assert torch.equal(place, got)
    c.check_grads(adapt_grad(c.y.to(DEV), *c.on(DEV), tp, shard, wide=True, **c.how(DEV)), c.y, True)


@gpu
def test_fp16_sums_of_the_smallest_values():
    """g and u below fp16's and near fp32's smallest normal values still reach a wide gradient."""
    note("adapt fp16 smallest")
    c = Case("fp16", 1, 136, 264, 40, 2, 8, run=5, sigma=2.0 ** -13)
    c.scale = torch.tensor([2.0 ** -100, 2.0 ** -101])
    got = adapt_grad(c.y.to(DEV), *c.on(DEV), 1, 136, wide=True, need=(False, True, True), **c.how(DEV))
    c.check_grads((None, *got[1:]), c.y, True, need=(False, True, True))


@gpu
@pytest.mark.parametrize("m", [5, 90])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_index_types_and_no_scale(m, index):
    note(f"adapt index {m} {index}")
    c = Case("bf16", 2, 136, 264, m, 4, 16, scaled=False, index=index)
    c.check(adapt(c.y.to(DEV), *c.on(DEV), 2, 136))
    c.check_grads(adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136), c.y)
    one = Case("bf16", 1, 136, 264, m, 4, 16, scaled=False, index=index)
    c2 = adapt(one.y[0].to(DEV), *one.on(DEV), 1, 136)
    assert c2.shape == (m, 136)
    one.check(c2[None])


@gpu
@pytest.mark.parametrize("m", [7, 64, 100])
def test_nothing_to_add(m):
    note(f"adapt nothing {m}")
    c = Case("fp16", 2, 72, 136, m, 3, 8, left_out=1.1)
    got = adapt(c.y.to(DEV), *c.on(DEV), 2, 72, **c.how(DEV))
    assert torch.equal(got.cpu(), c.y)
    for t in adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 72, **c.how(DEV)):
        assert not t.any()


@gpu
def test_no_rows():
    c = Case("bf16", 2, 72, 136, 0, 3, 8)
    assert adapt(c.y.to(DEV), *c.on(DEV), 2, 72, **c.how(DEV)).shape == (2, 0, 72)
    dx, da, db = adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 72, **c.how(DEV))
    assert dx.shape == (0, 136) and not da.any() and not db.any()


@gpu
@pytest.mark.parametrize("m", [40, 200])
def test_values_of_others_reach_no_row(m):
    """Infinities and NaN in an adapter, in x of rows without one and in one row's x and dy stay with their own."""
    note(f"adapt poison {m}")
    c = Case("bf16", 2, 136, 264, m, 4, 16)
    c.index[: m // 2] = torch.arange(m // 2) % 4
    clean = [t.clone() for t in (c.x, c.a, c.b)]
    bad = 2
    c.a[bad], c.b[bad] = math.nan, math.inf
    own = (c.index == bad)
    bare = (c.index < 0) | (c.index > 3)
    c.x[bare] = math.inf
    c.index[1], own[1] = 1, False
    lone = torch.zeros(m, dtype=torch.bool)
    lone[1] = True
    c.x[1] = math.nan
    y = c.y.clone()
    y[:, 0, 5] = math.nan
    got = adapt(y.to(DEV), *c.on(DEV), 2, 136, **c.how(DEV)).cpu()
    assert torch.equal(got[:, bare].view(torch.int16), y[:, bare].view(torch.int16))
    assert got[:, lone].isnan().all() and not got[:, own].isfinite().any()
    c.x, c.a, c.b = clean
    rest = ~(bare | own | lone)
    rest[0] = False
    want, bound = oa.adapt_bound(c.flat(c.y), *c.low(), "bf16")
    got = c.flat(got)
    assert (np.abs(got - want) <= bound)[rest.numpy()].all()


@gpu
@pytest.mark.parametrize("m", [40, 200])
def test_gradients_of_others_stay_theirs(m):
    note(f"adapt grad poison {m}")
    c = Case("bf16", 2, 136, 264, m, 4, 16, sigma=0.1)
    c.index[: m // 2] = torch.arange(m // 2) % 4
    own, bare = c.index == 2, (c.index < 0) | (c.index > 3)
    dy, x = c.y.clone(), c.x.clone()
    wants = adapt_grad(dy.to(DEV), *c.on(DEV), 2, 136, **c.how(DEV))
    dy[:, own], c.x[bare] = math.inf, math.nan
    dy[:, bare] = math.nan
    c.x[own] = math.nan
    got = adapt_grad(dy.to(DEV), *c.on(DEV), 2, 136, **c.how(DEV))
    keep = torch.tensor([0, 1, 3])
    assert torch.equal(got[0].cpu()[~own], wants[0].cpu()[~own])
    assert torch.equal(got[1].cpu()[keep], wants[1].cpu()[keep])
    assert torch.equal(got[2].cpu()[keep], wants[2].cpu()[keep])
    assert not got[1][2].isfinite().any() and not got[2][2].isfinite().any()
    c.x = x


@gpu
def test_fp16_of_any_size():
    """fp16's low-rank values far outside of its range on the way to a result inside."""
    note("adapt fp16 range")
    for up, down in ((100.0, 2.0 ** -14), (2.0 ** -10, 64.0)):
        c = Case("fp16", 2, 136, 1032, 90, 3, 16, sigma=1e-3, run=7)
        c.x = (c.x * up).half()
        c.a = (c.a * 30 * up).half()
        c.b = (c.b * down).half()
        c.check(adapt(c.y.to(DEV), *c.on(DEV), 2, 136, **c.how(DEV)))
        c.check_grads(adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136, wide=True, **c.how(DEV)), c.y, True)


@gpu
@pytest.mark.parametrize("m,n,rank", [(40, 4, 32), (40, 4, 40), (56, 3, 24), (57, 4, 8), (300, 3, 64), (1100, 40, 24)])
def test_fp16_gradients_of_small_and_large_adapters(m, n, rank):
    """Each adapter within what its own rows alone allow, the others' however large."""
    note(f"adapt fp16 sizes {m} {n} {rank}")
    c = Case("fp16", 2, 136, 264, m, n, rank, run=3)
    c.scale = c.scale * 2.0 ** torch.tensor([8.0 if i % 2 else -14.0 for i in range(n)])
    dx, da, db = adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136, wide=True, **c.how(DEV))
    c.check_grads((dx, da, db), c.y, True)
    dy, (x, a, b, index, scale) = c.flat(c.y), c.low()
    for i in range(n):
        rows = np.flatnonzero(index == i)
        _, bounds = oa.adapt_grad_bound(dy[rows], x[rows], a[i:i + 1], b[i:i + 1], np.zeros(len(rows), int), scale[i:i + 1],
                                        "fp16", "fp32")
        wants = oa.adapt_grad(dy[rows], x[rows], a[i:i + 1], b[i:i + 1], np.zeros(len(rows), int), scale[i:i + 1])
        for got, want, bound in zip((f64(da[i]), f64(db[i])), wants[1:], bounds[1:]):
            assert (np.abs(got - want[0]) <= bound[0]).all(), (i, np.max(np.abs(got - want[0]) / (bound[0] + 1e-300)))


@gpu
@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("dtype,m,rank", [("fp16", 30, 16), ("fp16", 30, 72), ("bf16", 30, 16), ("bf16", 300, 16),
                                          ("bf16", 300, 40), ("fp16", 300, 16)])
def test_gradients_that_are_not_needed_of_any_form(dtype, m, rank, need):
    note(f"adapt need {dtype} {m} {rank} {need}")
    c = Case(dtype, 2, 136, 264, m, 4, rank, run=2)
    c.check_grads(adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136, need=need, **c.how(DEV)), c.y, need=need)


@gpu
@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (True, True, False)])
def test_gradients_that_are_not_needed(need):
    note(f"adapt need {need}")
    c = Case("bf16", 2, 136, 264, 70, 4, 16, sigma=0.1)
    got = adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136, need=need, **c.how(DEV))
    c.check_grads(got, c.y, need=need)
    with pytest.raises(ValueError):
        adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 136, need=(False,) * 3)


@gpu
@pytest.mark.parametrize("m", [9, 150])
def test_autograd(m):
    note(f"adapted {m}")
    c = Case("bf16", 2, 136, 264, m, 4, 16, run=3)
    x, a, b, index = c.on(DEV)
    y = c.y.to(DEV)
    leaves = [t.requires_grad_() for t in (y, x, a, b)]
    out = adapted(y, x, a, b, index, 2, 136, **c.how(DEV))
    c.check(out)
    dy = (torch.randn(c.y.shape, generator=torch.Generator().manual_seed(9)) * 0.1).to(torch.bfloat16)
    out.backward(dy.to(DEV))
    assert torch.equal(y.grad.cpu(), dy)
    c.check_grads([t.grad for t in leaves[1:]], dy)
    a.requires_grad_(False)
    for t in leaves:
        t.grad = None
    adapted(y, x, a, b, index, 2, 136, **c.how(DEV)).float().sum().backward()  # an expanded gradient
    assert a.grad is None
    c.check_grads((x.grad, None, b.grad), torch.ones_like(c.y), need=(True, False, True))
    with pytest.raises(ValueError):
        adapted(y, x, a, b, index, 2, 136, scale=torch.ones(4, device=DEV, requires_grad=True))


@gpu
def test_repeats_its_bits_on_any_stream():
    note("adapt repeat")
    for m in (50, 500):
        c = Case("bf16", 4, 1000, 520, m, 9, 24, run=5)
        args = (c.y.to(DEV), *c.on(DEV), 4, 1000)
        first = [adapt(*args, **c.how(DEV)), *adapt_grad(*args, **c.how(DEV))]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = [adapt(*args, **c.how(DEV)), *adapt_grad(*args, **c.how(DEV))]
        side.synchronize()
        for a, b in zip(first, second):
            assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("m", [33, 300])
def test_captured_calls(m):
    note(f"adapt graph {m}")
    c = Case("fp16", 2, 264, 520, m, 5, 16, run=2, sigma=0.1)
    x, a, b, index = c.on(DEV)
    y = c.y.to(DEV)
    adapt(y, x, a, b, index, 2, 264, **c.how(DEV)), adapt_grad(y, x, a, b, index, 2, 264, **c.how(DEV))
    how = c.how(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = adapt(y, x, a, b, index, 2, 264, **how)
        grads = adapt_grad(y, x, a, b, index, 2, 264, **how)
    for seed in (2, 3, 4):
        c = Case("fp16", 2, 264, 520, m, 5, 16, run=seed, sigma=0.1, seed=seed)
        for t, v in ((x, c.x), (a, c.a), (b, c.b), (index, c.index), (y, c.y), (how["scale"], c.scale)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out)
        c.check_grads(grads, c.y)
        again = [adapt(y, x, a, b, index, 2, 264, **how), *adapt_grad(y, x, a, b, index, 2, 264, **how)]
        for p, q in zip([out, *grads], again):
            assert torch.equal(p, q)


@gpu
def test_captured_autograd():
    note("adapted graph")
    c = Case("bf16", 2, 136, 264, 70, 4, 16, run=3)
    x, a, b, index = c.on(DEV)
    y, how = c.y.to(DEV), c.how(DEV)
    dy = (torch.randn(c.y.shape, generator=torch.Generator().manual_seed(9)) * 0.1).to(torch.bfloat16).to(DEV)

    def step(leaves):
        return torch.autograd.grad(adapted(*leaves, index, 2, 136, **how), leaves, dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step([t.detach().requires_grad_() for t in (y, x, a, b)])
    torch.cuda.current_stream().wait_stream(side)
    leaves = [t.detach().requires_grad_() for t in (y, x, a, b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(leaves)
    for seed in (5, 6, 7):
        c = Case("bf16", 2, 136, 264, 70, 4, 16, run=seed, seed=seed)
        with torch.no_grad():
            for t, v in zip((*leaves, index, how["scale"]), (c.y, c.x, c.a, c.b, c.index, c.scale)):
                t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        c.check_grads(got[1:], dy.cpu())
        for p, q in zip(got, step([t.detach().requires_grad_() for t in leaves])):
            assert torch.equal(p, q)


@gpu
def test_past_32_bit_offsets():
    rows, vocab = 14000, 163840  # y and dy are 4.6 GB
    note("adapt 4.6 GB")
    c = Case("bf16", 8, 20480, 264, 48, 3, 8, run=5, sigma=0.1)
    y = torch.zeros(8, rows, 20480, dtype=torch.bfloat16, device=DEV)
    y[:, -48:] = c.y.to(DEV)
    x = torch.zeros(rows, 264, dtype=torch.bfloat16, device=DEV)
    x[-48:] = c.x.to(DEV)
    index = torch.full((rows,), 1, dtype=torch.int64, device=DEV)
    index[-48:] = c.index.to(DEV)
    _, a, b, _ = c.on(DEV)
    dx, da, db = adapt_grad(y, x, a, b, index, 8, 20480, **c.how(DEV))
    c.check_grads((dx[-48:], da, db), c.y)
    assert not dx[:-48].any()
    adapt(y, x, a, b, index, 8, 20480, out=y, **c.how(DEV))
    c.check(y[:, -48:])
    assert not y[:, :-48].any()


@gpu
@pytest.mark.parametrize("dtype,rank", [("bf16", 64), ("bf16", 136), ("fp16", 16), ("fp16", 40)])
def test_larger_than_the_caches(dtype, rank):
    rows, tail = 900, 40  # y and dy are 295 MB
    note(f"adapt 295 MB {dtype} {rank}")
    c = Case(dtype, 8, 20480, 136, tail, 3, rank, run=7, sigma=0.1)
    y = torch.zeros(8, rows, 20480, dtype=DT[dtype], device=DEV)
    y[:, -tail:] = c.y.to(DEV)
    x = torch.zeros(rows, 136, dtype=DT[dtype], device=DEV)
    x[-tail:] = c.x.to(DEV)
    index = torch.full((rows,), 1, dtype=torch.int64, device=DEV)
    index[-tail:] = c.index.to(DEV)
    _, a, b, _ = c.on(DEV)
    dx, da, db = adapt_grad(y, x, a, b, index, 8, 20480, **c.how(DEV))
    c.check_grads((dx[-tail:], da, db), c.y)
    assert not dx[:-tail].any()
    out = adapt(y, x, a, b, index, 8, 20480, **c.how(DEV))
    c.check(out[:, -tail:])
    assert not out[:, :-tail].any()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [1, 20, 300])
def test_most_adapters(m, dtype):
    note(f"adapt 32768 adapters {m} {dtype}")
    c = Case(dtype, 2, 8, 16, m, 1 << 15, 8, run=2)
    c.index[0], c.index[-1] = (1 << 15) - 1, 1 << 15  # the last one, and none
    c.check(adapt(c.y.to(DEV), *c.on(DEV), 2, 8, **c.how(DEV)))
    c.check_grads(adapt_grad(c.y.to(DEV), *c.on(DEV), 2, 8, **c.how(DEV)), c.y)


@gpu
def test_two_graphs_at_once():
    note("adapt two graphs")
    cases = [Case("bf16", 2, 1000, 520, 300, 3, 24, run=40), Case("fp16", 3, 328, 264, 50, 7, 16, run=2)]
    graphs = []
    for c in cases:
        args, how = (c.y.to(DEV), *c.on(DEV), c.tp, c.shard), c.how(DEV)
        eager = [adapt(*args, **how), *adapt_grad(*args, **how)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [adapt(*args, **how), *adapt_grad(*args, **how)]
        graphs.append((graph, eager, got, args, how))
    sides = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for _, _, got, _, _ in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for side, (graph, _, _, args, how) in zip(sides, graphs):
            with torch.cuda.stream(side):
                for _ in range(8):
                    graph.replay()
        again = [adapt(*args, **how) for _, _, _, args, how in graphs]  # beside the replays
        torch.cuda.synchronize()
        for (_, eager, got, _, _), other in zip(graphs, again):
            assert torch.equal(other, eager[0])
            for p, q in zip(got, eager):
                assert torch.equal(p, q)


@gpu
def test_wrong_workspaces_and_overlaps_are_refused():
    c = Case("bf16", 2, 72, 136, 9, 3, 8)
    y = c.y.to(DEV)
    room = torch.zeros(y.numel() + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(HgError):
        adapt(room[:-8].view(y.shape), *c.on(DEV), 2, 72, out=room[8:].view(y.shape))
    with pytest.raises(ValueError):
        adapt(y, *c.on(DEV), 2, 72, out=y.float())
