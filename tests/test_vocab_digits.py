"""How many digits the cross entropy keeps: of logits that are long sums of one
sign, by the rms of its losses' errors over rows that lean to their labels; of
gradients, against the rounding of the result alone."""

from __future__ import annotations

import math

import pytest
import torch

from tp_vocab_logits_amd import vocab_train as vt

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U32 = 2.0 ** -24


def leaning(vocab, hidden, m, dtype, seed):
    """Rows whose label's logit is 0.8 to 1.1 log(vocab), a sum of terms mostly
    of one sign, beside logits of about 1.7; the matrix, labels, and in 64 bits
    the losses and the rms of the labels' logits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn(vocab, hidden, generator=g, device=DEV) * 0.02).to(DT[dtype])
    labels = torch.randint(0, vocab, (m,), generator=g, device=DEV)
    lean = (0.8 + 0.3 * torch.rand(m, 1, generator=g, device=DEV)) * math.log(vocab) / (0.02 ** 2 * hidden)
    x = (torch.randn(m, hidden, generator=g, device=DEV) + lean * w[labels].float()).to(DT[dtype])
    z = torch.cat([x.double() @ w[a:a + 16384].double().t() for a in range(0, vocab, 16384)], dim=1)
    target = z.gather(1, labels[:, None]).squeeze(1)
    return x, w, labels, torch.logsumexp(z, 1) - target, float(target.square().mean().sqrt())


def rms_error(loss, want):
    return float((loss.double() - want).square().mean().sqrt())


# A sum that grows to Z in n additions, each rounded to half a step at most
# (uniformly: U/sqrt(3) rms, U = 2^-24 of the size reached), is off by about
# Z U sqrt(n) / 3. The matrix cores round at least once per 32 products, so one
# chain of 7168 products has 224 roundings or more and is off by 5 Z U. In chains
# of 1024, the chains' own roundings are at a seventh of the size: with a rounding
# per 4 products, 256 in each of seven chains, sqrt(7 * 256) / 3 / 7 = 2 Z U, and
# the seven additions of the chains 0.95 Z U: 2.2 together; 1 with a rounding per
# 32. What follows (the exponentials, the logarithm, one rounding of the loss) is
# of the size of U alone. Less than 3 Z U therefore, which one chain is not.
SPLIT_CHAINS = 3.0
# One chain with a rounding per 8 products: sqrt(896) / 3.
ONE_CHAIN = 10.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [13, 32, 50, 128])
@pytest.mark.parametrize("tp,shard", [(8, 8256), (2, 22240), (4, 4064)])
def test_few_rows_keep_the_digits_of_long_sums(tp, shard, m, dtype):
    """V = 66048: runs of more than 128 entries per workgroup; 44480 and 16256:
    runs that fill a stage with two and four chunks of k."""
    print(f"[gpu] digits {tp=} {shard=} {m=} {dtype}", flush=True)
    x, w, labels, want, size = leaning(tp * shard, 7168, m, dtype, m)
    loss, lse = vt.head_xent(x, w, labels, tp, shard)
    assert rms_error(loss, want) <= SPLIT_CHAINS * U32 * size
    apart = [b.clone() for b in w.view(tp, shard, -1)]  # blocks that do not follow one another
    again = vt.head_xent(x, apart, labels, tp, shard)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("vocab,m", [(8192, 40), (8192, 200), (66048, 1), (66048, 128)])
def test_a_small_step_keeps_the_digits_of_long_sums(vocab, m, dtype):
    print(f"[gpu] digits of a small step {vocab=} {m=} {dtype}", flush=True)
    x, w, labels, want, size = leaning(vocab, 7168, m, dtype, 1)
    loss = vt.head_xent_step(x, w, labels, torch.ones(m, device=DEV), 1, vocab)[0]
    assert rms_error(loss, want) <= SPLIT_CHAINS * U32 * size


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_rows_are_off_by_one_chain(dtype):
    """The 256 x 256 tile sums a logit in one chain: no more than that."""
    print(f"[gpu] digits of many rows {dtype}", flush=True)
    x, w, labels, want, size = leaning(66048, 7168, 300, dtype, 2)
    loss = vt.head_xent(x, w, labels, 8, 8256)[0]
    assert rms_error(loss, want) <= ONE_CHAIN * U32 * size


HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def gradients(x, w, labels, grad, vocab):
    """In 64 bits."""
    kept = labels >= 0
    xd, wd = torch.where(kept[:, None], x.double(), 0.0), w[:vocab].double()
    d = torch.softmax(xd @ wd.t(), dim=1)
    d[torch.nonzero(kept).squeeze(1), labels[kept]] -= 1.0
    d *= torch.where(kept, grad.double(), 0.0)[:, None]
    dw = torch.zeros(w.shape, dtype=torch.float64, device=DEV)
    dw[:vocab] = d.t() @ xd
    return d @ wd, dw


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


# m, rows of the matrix, hidden, vocabulary, limit of the workspace: small tiles,
# big ones, sums split over the vocabulary and over the rows, the vocabulary in
# pieces, more labels than one turn lists and more in a tile than one step takes
GRADIENTS = [(1, 2048, 64, 2048, 0), (33, 2048, 264, 2001, 0), (300, 17408, 520, 17001, 0),
             (3000, 2048, 1032, 2047, 0), (6000, 1024, 136, 1000, 0), (700, 8192, 264, 8190, 6 << 20)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("often", [0.0, 0.5])
@pytest.mark.parametrize("m,rows,hidden,vocab,limit", GRADIENTS)
def test_a_gradient_is_rounded_once(m, rows, hidden, vocab, limit, often, dtype):
    """The label's d is rounded to 16 bits for the products and would be off by
    up to half a step, which is as much as the result's own rounding, on the
    one large term of a row of dX and of dW. What the rounding leaves out is
    added, so the other terms' roundings are left. Probabilities here are about
    1/vocab each: their errors, half a step of each at random signs, sum up to
    vocab^-1/2 <= 1/30 of what the label's would be (with the label's term 1, a
    row of dX has vocab others of 1/vocab; a row of dW has m, on vocab rows). The
    rounding of the result may thus be exceeded by a thousandth, and 10 % is
    allowed; in fp32, a tenth of half a step."""
    print(f"[gpu] gradients {m=} {rows=} {hidden=} {vocab=} {often=} {dtype}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(m + vocab)
    x = torch.randn(m, hidden, generator=g, device=DEV).to(DT[dtype])
    w = (torch.randn(rows, hidden, generator=g, device=DEV) * 0.4 / hidden ** 0.5).to(DT[dtype])
    labels = torch.randint(0, vocab, (m,), generator=g, device=DEV)
    labels[torch.rand(m, generator=g, device=DEV) < often] = vocab - 3
    grad = 0.5 + torch.rand(m, generator=g, device=DEV)
    if m > 1:
        labels[torch.rand(m, generator=g, device=DEV) < 0.1] = -100
    want_x, want_w = gradients(x, w, labels, grad, vocab)
    _, lse, dx, dw = vt.head_xent_step(x, w, labels, grad, 2, rows // 2, vocab=vocab, workspace_limit=limit)
    later = vt.head_xent_grad(x, w, labels, lse, grad, 2, rows // 2, vocab=vocab, workspace_limit=limit)
    wide = vt.head_xent_step(x, w, labels, grad, 2, rows // 2, vocab=vocab, workspace_limit=limit,
                             dw=torch.empty(rows, hidden, device=DEV))[3]
    for got, want in ((dx, want_x), (dw, want_w), (later[0], want_x), (later[1], want_w)):
        assert off(got, want) <= 1.1 * off(want.to(DT[dtype]), want)
    assert off(wide, want_w) <= 0.1 * HALF_STEP[dtype]
