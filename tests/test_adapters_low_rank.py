"""The low-rank values of the adapters on their way to a result: sums that come out exact in fp32, so that nothing but
what the second product makes of them is left; infinities and adapters of different size (GPU). And that the oracle's
bounds see a mistake there (CPU).

Every row has one entry on the side that is summed first, so u (or g) is one product of two 16-bit numbers, at most 22
bits, and a factor: off by 2^-24 of itself. An entry of the result is then one product with a 16-bit number, in up to
three pieces that fp32 adds up, each within 2^-23 (a sum that cuts off): 2^-24 + 3 * 2^-23 < 2^-21 in all. What fp16
holds of a value ends 2^-38 below the largest of its row, or of its adapter's rows."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import adapters as oa
from tp_vocab_logits_amd import _lib, adapt, adapt_grad

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half of the smallest step of a 16-bit result
SUMS = 2.0 ** -21
gpu = pytest.mark.gpu

# rows, adapters, rank: few rows; many of many adapters; many of few (the streaming form), up to 16, 64 and more ranks
FORMS = [(5, 3, 8), (40, 4, 32), (64, 2, 72), (90, 9, 16), (150, 20, 64), (200, 2, 72), (300, 2, 16), (300, 3, 40), (200, 1, 64)]
TP, SHARD, HIDDEN = 2, 136, 264
V = TP * SHARD


def note(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)


def f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, dtype, m, n, rank, seed):
        g = torch.Generator().manual_seed(1000 * seed + m + rank)
        self.g, self.kind, self.t, self.m = g, dtype, DT[dtype], m
        self.index = torch.randint(0, n, (m,), generator=g)
        self.scale = torch.rand(n, generator=g) + 0.5
        self.a = (torch.randn(n, rank, HIDDEN, generator=g)).to(self.t)
        self.b = (torch.randn(n, V, rank, generator=g)).to(self.t)
        self.sizes = 2.0 ** -torch.randint(0, 10, (m, 1), generator=g)  # rows of different size
        self.turn = torch.empty(m, dtype=torch.long)  # which of its adapter's rows a row is
        for i in range(n):
            rows = torch.nonzero(self.index == i).squeeze(1)
            self.turn[rows] = torch.arange(len(rows))
        self.most = int(self.turn.max()) + 1

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def one_entry(self, width):
        """[m, width]: one entry a row."""
        out = torch.zeros(self.m, width)
        at = torch.randint(0, width, (self.m, 1), generator=self.g)
        return out.scatter_(1, at, self.randn(self.m, 1) * self.sizes).to(self.t)

    def in_turn(self, width):
        """[m, width]: an adapter's rows have their entries in different columns (as far as there are columns)."""
        mine = torch.arange(width)[None, :] % self.most == self.turn[:, None]
        return (self.randn(self.m, width) * mine).to(self.t)

    def shards(self, flat):
        return flat.view(self.m, TP, SHARD).transpose(0, 1).contiguous()

    def on(self):
        return [t.to(DEV) for t in (self.a, self.b, self.index)]

    def largest(self, low):
        """Of each adapter's rows."""
        return np.array([np.abs(low[self.index.numpy() == i]).max(initial=0.0) for i in range(len(self.scale))])


def test_bounds_are_each_adapters_own():
    """fp16's pieces, emulated: by each adapter's largest value they are within the bounds, by the call's they are not."""
    rng = np.random.RandomState(0)
    index, x, dy = rng.randint(0, 2, 40), rng.randn(40, 24), rng.randn(40, 16)
    a, b, scale = rng.randn(2, 8, 24), rng.randn(2, 16, 8), np.array([2.0 ** 20, 2.0 ** -20])
    (_, _, want), (_, _, bound) = oa.adapt_grad_bound(dy, x, a, b, index, scale, "fp16", "fp32")
    us = [scale[i] * (x[index == i] @ a[i].T) for i in range(2)]
    for tops, good in (([np.abs(u).max() for u in us], True), ([max(np.abs(u).max() for u in us)] * 2, False)):
        within = []
        for i, (u, top) in enumerate(zip(us, tops)):
            factor, held = 2.0 ** (13 - np.floor(np.log2(top))), np.zeros_like(u)
            for _ in range(3):
                held += (u * factor - held).astype(np.float16)
            within.append((np.abs(dy[index == i].T @ (held / factor) - want[i]) <= bound[i]).all())
        assert all(within) == good


def near(got, want, bound):
    e = np.abs(got - want)
    assert (e <= bound).all(), np.max(e / bound)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,rank", FORMS)
def test_wide_gradients_hold_what_fp32_does(dtype, m, n, rank):
    note(f"adapt wide {dtype} {m} {n} {rank}")
    c = Case(dtype, m, n, rank, 1)
    floor = 0.0 if dtype == "bf16" else 2.0 ** -38
    index, scale = c.index.numpy(), f64(c.scale)
    # db: u of one entry of x
    x, dy = c.one_entry(HIDDEN), c.in_turn(V)
    a, b, i = c.on()
    _, _, db = adapt_grad(c.shards(dy).to(DEV), x.to(DEV), a, b, i, TP, SHARD, scale=c.scale.to(DEV), wide=True,
                          need=(False, False, True))
    u = scale[index][:, None] * np.einsum("mh,mrh->mr", f64(x), f64(c.a)[index])
    parts = np.einsum("mv,mr->mvr", f64(dy), u)
    want, size, other = np.zeros((n, V, rank)), np.zeros((n, V, rank)), np.zeros((n, V))
    np.add.at(want, index, parts)
    np.add.at(size, index, np.abs(parts))
    np.add.at(other, index, np.abs(f64(dy)))
    # (where two rows share a column, their sum: the bound is of what is added)
    near(f64(db), want, SUMS * size + floor * c.largest(u)[:, None, None] * other[:, :, None] + 2.0 ** -140)
    # da: g of one entry of dy
    dy, x = c.one_entry(V), c.in_turn(HIDDEN)
    _, da, _ = adapt_grad(c.shards(dy).to(DEV), x.to(DEV), a, b, i, TP, SHARD, scale=c.scale.to(DEV), wide=True,
                          need=(False, True, False))
    g = scale[index][:, None] * np.einsum("mv,mvr->mr", f64(dy), f64(c.b)[index])
    parts = np.einsum("mr,mh->mrh", g, f64(x))
    want, size, other = np.zeros((n, rank, HIDDEN)), np.zeros((n, rank, HIDDEN)), np.zeros((n, HIDDEN))
    np.add.at(want, index, parts)
    np.add.at(size, index, np.abs(parts))
    np.add.at(other, index, np.abs(f64(x)))
    near(f64(da), want, SUMS * size + floor * c.largest(g)[:, None, None] * other[:, None, :] + 2.0 ** -140)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,rank", FORMS)
def test_what_cancels_is_fp32s(dtype, m, n, rank):
    """y takes nearly all of what the adapter adds away; the rounding is the small result's own."""
    note(f"adapt cancel {dtype} {m} {n} {rank}")
    c = Case(dtype, m, n, rank, 2)
    x = c.one_entry(HIDDEN)
    mine = torch.randint(0, rank, (n, V, 1), generator=c.g)
    c.b = c.b * (torch.arange(rank)[None, None, :] == mine)  # one rank a column
    a, b, i = c.on()
    index, scale = c.index.numpy(), f64(c.scale)
    u = scale[index][:, None] * np.einsum("mh,mrh->mr", f64(x), f64(c.a)[index])
    more = np.einsum("mvr,mr->mv", f64(c.b)[index], u)
    y = (-torch.from_numpy(more)).to(c.t)
    got = adapt(c.shards(y).to(DEV), x.to(DEV), a, b, i, TP, SHARD, scale=c.scale.to(DEV))
    got = f64(got.transpose(0, 1).reshape(m, V))
    want = f64(y) + more
    floor = 0.0 if dtype == "bf16" else 2.0 ** -38
    lost = SUMS * np.abs(more) + floor * np.abs(u).max(axis=1, keepdims=True) * np.abs(f64(c.b)).max()
    near(got, want, lost + HALF_STEP[dtype] * (np.abs(want) + lost) + LEAST[dtype])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,rank", FORMS)
def test_input_gradients_that_cancel(dtype, m, n, rank):
    """Two ranks that all but cancel in dx: g_0 = big + small, g_1 = big, a_1 = -a_0."""
    note(f"adapt dx cancel {dtype} {m} {n} {rank}")
    c = Case(dtype, m, n, rank, 3)
    c.a = torch.zeros_like(c.a)
    c.a[:, 0] = c.randn(n, HIDDEN).to(c.t)
    c.a[:, rank - 1] = -c.a[:, 0]
    c.b = torch.zeros_like(c.b)
    # integers of up to 8 and 4 bits: big <= 2^16 and small are one fp32 sum that is exact
    c.b[:, 3, 0] = c.b[:, 3, rank - 1] = torch.randint(128, 256, (n,), generator=c.g).to(c.t)
    c.b[:, 140, 0] = torch.randint(1, 16, (n,), generator=c.g).to(c.t)
    dy = torch.zeros(m, V)
    dy[:, 3] = torch.randint(128, 256, (m,), generator=c.g).float()
    dy[:, 140] = 1.0
    dy = dy.to(c.t)
    a, b, i = c.on()
    dx, _, _ = adapt_grad(c.shards(dy).to(DEV), torch.zeros(m, HIDDEN, dtype=c.t, device=DEV), a, b, i, TP, SHARD,
                          scale=c.scale.to(DEV), need=(True, False, False))
    index = c.index.numpy()
    g = f64(c.scale)[index][:, None] * np.einsum("mv,mvr->mr", f64(dy), f64(c.b)[index])
    want = np.einsum("mr,mrh->mh", g, f64(c.a)[index])
    # g within 2^-24; up to six pieces of at most |g| |a| each, added within 2^-23
    lost = 6.5 * 2.0 ** -23 * np.einsum("mr,mrh->mh", np.abs(g), np.abs(f64(c.a)[index]))
    near(f64(dx), want, lost + HALF_STEP[dtype] * (np.abs(want) + lost) + LEAST[dtype])


@gpu
@pytest.mark.parametrize("m,n,rank", [(5, 3, 8), (90, 9, 16), (300, 2, 16), (200, 1, 64), (200, 2, 72)])
def test_low_rank_values_between_bf16s_largest_and_fp32s(m, n, rank):
    """A u that bf16 would round to infinity, and a factor that brings the result back."""
    note(f"adapt near fp32's largest {m} {n} {rank}")
    c = Case("bf16", m, n, rank, 4)
    top = 2.0 ** 127
    c.scale = torch.full((n,), (2.0 - 2.0 ** -12) * top)  # above bf16's largest, (2 - 2^-7) 2^127
    x = torch.zeros(m, HIDDEN, dtype=c.t)
    x[:, 5] = 1.0
    c.a = torch.zeros_like(c.a)
    c.a[:, 0, 5] = 1.0
    c.b = (c.b * 2.0 ** -126).to(c.t)
    a, b, i = c.on()
    y = torch.zeros(TP, m, SHARD, dtype=c.t, device=DEV)
    got = adapt(y, x.to(DEV), a, b, i, TP, SHARD, scale=c.scale.to(DEV))
    got = f64(got.transpose(0, 1).reshape(m, V))
    want = f64(c.b)[c.index.numpy()][:, :, 0] * f64(c.scale)[0]
    # bf16's smallest normal b is 2^-126: what lies below it may count as nothing
    small = np.abs(f64(c.b)[c.index.numpy()][:, :, 0]) < 2.0 ** -126
    near(np.where(small, want, got), want, (HALF_STEP["bf16"] + 2 * SUMS) * np.abs(want) + 1e-30)


@gpu
@pytest.mark.parametrize("m,n,rank", FORMS)
def test_fp16_adapters_go_by_their_own_largest(m, n, rank):
    """Adapters 2^40 apart: by one factor for all of them the small ones would be nothing."""
    note(f"adapt fp16 apart {m} {n} {rank}")
    n += n == 1
    c = Case("fp16", m, n, rank, 5)
    c.scale = c.scale * 2.0 ** torch.tensor([20.0 if i % 2 else -20.0 for i in range(n)])
    dy, x = (c.randn(m, w).to(c.t) for w in (V, HIDDEN))
    a, b, i = c.on()
    got = adapt_grad(c.shards(dy).to(DEV), x.to(DEV), a, b, i, TP, SHARD, scale=c.scale.to(DEV), wide=True,
                     need=(False, True, True))
    wants, bounds = oa.adapt_grad_bound(f64(dy), f64(x), f64(c.a), f64(c.b), c.index.numpy(), f64(c.scale), "fp16", "fp32")
    for t, want, bound in zip(got[1:], wants[1:], bounds[1:]):
        near(f64(t), want, bound + 1e-300)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,rank", [(40, 4, 16), (56, 3, 32), (57, 3, 32), (40, 4, 40), (200, 4, 16), (300, 3, 40), (200, 4, 72)])
def test_what_is_not_finite_stays_where_it_belongs(dtype, m, n, rank):
    """An adapter of infinities, rows of infinities that have it, rows without an adapter; then one rank of an adapter."""
    note(f"adapt not finite {dtype} {m} {n} {rank}")
    c = Case(dtype, m, n, rank, 6)
    c.index[::7] = -1
    c.index[:n] = torch.arange(n)
    own, bare = c.index == 1, c.index < 0
    y, dy, x = ((c.randn(m, w) * 0.1).to(c.t) for w in (V, V, HIDDEN))
    scale = c.scale.to(DEV)

    def run(y, dy, x, a, b):
        low = (x.to(DEV), a.to(DEV), b.to(DEV), c.index.to(DEV), TP, SHARD)
        out = adapt(c.shards(y).to(DEV), *low, scale=scale).transpose(0, 1).reshape(m, V)
        return [t.cpu() for t in (out, *adapt_grad(c.shards(dy).to(DEV), *low, scale=scale, wide=True))]

    clean = run(y, dy, x, c.a, c.b)
    a, b, bad_y, bad_dy, bad_x = c.a.clone(), c.b.clone(), y.clone(), dy.clone(), x.clone()
    a[1], b[1] = float("inf"), float("nan")
    bad_dy[own], bad_x[own], bad_dy[bare], bad_x[bare] = -float("inf"), float("inf"), float("nan"), float("nan")
    out, dx, da, db = run(bad_y, bad_dy, bad_x, a, b)
    others = torch.arange(n) != 1
    assert torch.equal(out[~own], clean[0][~own]) and torch.equal(dx[~own], clean[1][~own])
    assert torch.equal(da[others], clean[2][others]) and torch.equal(db[others], clean[3][others])
    assert not any(t.isfinite().any() for t in (out[own], dx[own], da[1], db[1]))
    # one rank of A: u's; the others' columns of dB are those of an adapter without it
    a, b = c.a.clone(), c.b.clone()
    a[1, 3] = float("inf")
    out, dx, da, db = run(y, dy, x, a, b)
    assert torch.equal(da, clean[2]) and not db[1, :, 3].isfinite().any() and not out[own].isfinite().any()
    a[1, 3] = 0.0
    low = (f64(x), f64(a), f64(b), c.index.numpy(), f64(c.scale))
    wants, bounds = oa.adapt_grad_bound(f64(dy), *low, dtype, "fp32")
    keep = np.arange(rank) != 3
    near(f64(db)[..., keep], wants[2][..., keep], bounds[2][..., keep] + 1e-300)
    # one rank of B: g's
    a, b = c.a.clone(), c.b.clone()
    b[1, 5, 3] = -float("inf")
    out, dx, da, db = run(y, dy, x, a, b)
    assert torch.equal(db, clean[3]) and not da[1, 3].isfinite().any() and not dx[own].isfinite().any()
    b[1, 5, 3] = 0.0
    low = (f64(x), f64(a), f64(b), c.index.numpy(), f64(c.scale))
    wants, bounds = oa.adapt_grad_bound(f64(dy), *low, dtype, "fp32")
    near(f64(da)[:, keep], wants[1][:, keep], bounds[1][:, keep] + 1e-300)


def test_every_shape_within_the_limits_is_taken():
    """As many rows and columns as the form without streaming has no single launch for."""
    n = ctypes.c_size_t()
    for kind in (_lib.HG_ADAPT_ADD, _lib.HG_ADAPT_GRAD):
        for tp, shard, hidden, m, adapters, rank in (
                (8, 20480, 7168, 212000, 4, 72), (8, 20480, 7168, 262144, 1, 128), (1, 8, 8, 1 << 24, 1, 256),
                (8, 20480, 7168, 1 << 20, 1 << 10, 16), (1, 8, 1 << 20, 1 << 24, 500, 64), (64, 1 << 17, 8, 1 << 17, 3, 256)):
            shape = _lib.AdaptShape(tp, shard, hidden, m, adapters, rank, _lib.HG_BF16, 8)
            assert _lib.lib().hg_adapt_workspace(shape, kind, n) == _lib.HG_OK, (tp, shard, hidden, m, adapters, rank)
    # gradients: adapters x strips of 64 columns x chunks of 64 ranks
    for tp, shard, hidden, adapters, rank, taken in (
            (1, 8, 64 * 64, 1 << 15, 256, False), (1, 8, 64 * 63, 1 << 15, 256, True), (64, 72, 8, 1 << 15, 72, False),
            (64, 64, 8, 1 << 15, 72, True), (1, 64 * 256, 8, 1 << 15, 64, False), (1, 64 * 255, 8, 1 << 15, 64, True)):
        shape = _lib.AdaptShape(tp, shard, hidden, 5, adapters, rank, _lib.HG_BF16, 8)
        assert (_lib.lib().hg_adapt_workspace(shape, _lib.HG_ADAPT_GRAD, n) == _lib.HG_OK) == taken, (tp, shard, hidden, adapters, rank)


@gpu
def test_more_rows_than_one_launch_covers():
    m, rank, n, hidden, v = 14_950_003, 72, 3, 8, 8  # 934376 tiles x 9 strips, above 2^23
    note("adapt 15 million rows")
    g = torch.Generator(device=DEV).manual_seed(3)
    y, x = (torch.randn(m, w, generator=g, device=DEV).bfloat16() for w in (v, hidden))
    a = torch.randn(n, rank, hidden, generator=g, device=DEV).bfloat16()
    b = torch.randn(n, v, rank, generator=g, device=DEV).bfloat16()
    index = torch.randint(-1, n, (m,), generator=g, device=DEV)
    got = adapt(y, x, a, b, index, 1, v)
    # sums of 8 and of 72 terms in three pieces: (8 + 216 + 8) steps of 2^-23, below 2^-15
    for at in range(0, m, 1 << 20):
        part = slice(at, at + (1 << 20))
        want, size = y[part].double(), torch.zeros_like(y[part], dtype=torch.float64)
        for i in range(n):
            mine = (index[part] == i)[:, None]
            xs, ai, bi = x[part].double(), a[i].double(), b[i].double()
            want += torch.where(mine, (xs @ ai.t()) @ bi.t(), 0.0)
            size += torch.where(mine, (xs.abs() @ ai.abs().t()) @ bi.abs().t(), 0.0)
        e = (got[part].double() - want).abs()
        lost = 2.0 ** -15 * size
        assert (e <= lost + HALF_STEP["bf16"] * (want.abs() + lost)).all(), at
        bare = index[part] < 0
        assert torch.equal(got[part][bare], y[part][bare])
