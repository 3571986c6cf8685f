"""Sizes that choose the kernels' other variants: more rows than one packing
launch takes, vocabularies of more tiles than one turn merges, lookups and
gradients of many rows (GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import vocab as ov
from test_vocab_train import DEV, DT, Problem, check_embed_grad, f64, rand
from tp_vocab_logits_amd import vocab_train as vt

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,left_out", [(4097, 0.0), (5003, 0.4), (4999, 1.0)])
def test_more_rows_than_one_packing_launch(m, left_out, dtype):
    print(f"[gpu] many rows {m=} {left_out=} {dtype}", flush=True)
    p = Problem(3, 96, 72, m, 270, dtype, left_out, scale=0.7, z_weight=0.01)
    x, w, t, g = p.on_gpu()
    x[t == -100] = float("nan")
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 3, 96, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)
    again = vt.head_xent(x, w, t, 3, 96, **p.how)
    p.check_loss(*again)
    dx, dw = vt.head_xent_grad(x, w, t, lse, g, 3, 96, **p.how)
    p.check_grads(dx, dw, lse_used=f64(lse))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [100, 200])
def test_more_tiles_than_one_turn_merges(m, dtype):
    """The joining kernel merges 128 tiles of a row at a time: of 128 columns up
    to 128 rows, of 256 beyond."""
    print(f"[gpu] many tiles {m=} {dtype}", flush=True)
    p = Problem(2, 17024, 72, m, 33999, dtype, 0.1, z_weight=0.01)
    x, w, t, g = p.on_gpu()
    loss, lse, dx, dw = vt.head_xent_step(x, w, t, g, 2, 17024, **p.how)
    p.check_loss(loss, lse)
    p.check_grads(dx, dw)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [1, 17, 33, 128])
@pytest.mark.parametrize("tp,shard,hidden,vocab", [(2, 33248, 136, 66001), (1, 44512, 72, 44490)])
def test_few_rows_of_a_large_vocabulary(tp, shard, hidden, vocab, m, dtype):
    """Runs of several tiles per workgroup, and two workgroups per CU."""
    print(f"[gpu] few rows {vocab=} {m=} {dtype}", flush=True)
    p = Problem(tp, shard, hidden, m, vocab, dtype, 0.1 if m > 4 else 0.0, scale=-1.5, z_weight=0.01)
    x, w, t, _ = p.on_gpu()
    w[vocab:] = float("nan")
    loss, lse = vt.head_xent(x, w, t, tp, shard, **p.how)
    p.check_loss(loss, lse)
    if tp > 1:
        p.blocks = True
        again = vt.head_xent(x, p.on_gpu()[1], t, tp, shard, **p.how)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tp,shard,hidden,n", [(3, 70, 72, 33001), (2, 40, 2056, 1100), (4, 40, 8232, 260), (1, 9, 4096, 700)])
@pytest.mark.parametrize("scale", [1.0, 11.313708])
def test_lookup_of_many_rows(tp, shard, hidden, n, dtype, scale):
    """More than 2^18 vectors of 16 bytes; rows that end inside a workgroup's
    four vectors per lane, and more rows than the grid has."""
    print(f"[gpu] lookup {tp=} {shard=} {hidden=} {n=} {dtype} {scale}", flush=True)
    assert n * hidden * (4 if dtype == "fp32" else 2) >= 16 << 18
    w = rand((tp * shard, hidden), 1.0, 7, dtype).to(DEV)
    tokens = torch.randint(-2, tp * shard + 2, (n,), generator=torch.Generator().manual_seed(n)).to(DEV)
    inside = (tokens >= 0) & (tokens < tp * shard)
    want = torch.where(inside[:, None], w[tokens.clamp(0, tp * shard - 1)].double() * float(np.float32(scale)), 0.0)
    got = vt.embed(tokens, w, tp, shard, scale)
    bound = (ov.HALF_STEP[dtype] + 2 * ov.U32) * want.abs() + 2.0 ** -25 * (dtype == "fp16")
    assert ((got.double() - want).abs() <= bound).all()
    assert torch.equal(vt.embed(tokens.int(), w, tp, shard, scale), got)
    blocks = [w.view(tp, shard, hidden)[r].clone() for r in range(tp)]
    assert torch.equal(vt.embed(tokens, blocks, tp, shard, scale), got)
    w.fill_(float("nan"))
    assert not vt.embed(torch.full_like(tokens, -1), w, tp, shard, scale).any()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_tokens_in_a_large_gradient(dtype):
    """Zeros of more than 32 MB are a launch of their own."""
    print(f"[gpu] few tokens, large gradient {dtype}", flush=True)
    tp, shard, hidden, n = 4, 16500, 264, 100
    tokens = torch.randint(-1, tp * shard, (n,), generator=torch.Generator().manual_seed(1))
    tokens[20:50] = tokens[3]
    tokens[-1] = tp * shard - 1
    dy = rand((n, hidden), 1.0, 11, dtype)
    check_embed_grad(tokens, dy, tp, shard, 2.0, dtype)
    check_embed_grad(tokens, dy, tp, shard, 2.0, dtype, old=rand((tp * shard, hidden), 1.0, 12, dtype))
    if dtype != "fp32":
        check_embed_grad(tokens, dy, tp, shard, 2.0, dtype, wide=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tp,shard,n", [(2, 2500, 70001), (4, 75000, 140003), (1, 40, 140003)])
def test_gradient_of_many_tokens(tp, shard, n, dtype):
    """More counts than one turn of the scan takes (n > 65536), and blocks of
    more than 64 positions (n > 131072); frequent tokens and tokens outside."""
    print(f"[gpu] many tokens {tp=} {shard=} {n=} {dtype}", flush=True)
    rows = tp * shard
    g = torch.Generator().manual_seed(n)
    rank = torch.exp(torch.rand(n, generator=g) * np.log(rows + 1)).long() - 1
    tokens = torch.where(torch.rand(n, generator=g) < 0.1, -1, (rank * 7919) % (rows + 1))
    dy = rand((n, 16), 1.0, 11, dtype)
    got = check_embed_grad(tokens, dy, tp, shard, 2.0, dtype)
    assert torch.equal(vt.embed_grad(tokens.int().to(DEV), dy.to(DEV), tp, shard, 2.0), got)
    check_embed_grad(tokens, dy, tp, shard, 0.5, dtype, old=rand((rows, 16), 1.0, 12, dtype))


@gpu
def test_gradients_of_two_backward_passes_add_up():
    print("[gpu] two backward passes", flush=True)
    p = Problem(2, 96, 64, 50, 150, left_out=0.2, scale=0.7, z_weight=0.02)
    x, w, t, g = p.on_gpu()
    x.requires_grad_(), w.requires_grad_()
    (vt.head_loss(x, w, t, 2, 96, **p.how) * g).sum().backward()
    lse = vt.head_xent(x.detach(), w.detach(), t, 2, 96, **p.how)[1]
    p.check_grads(x.grad, w.grad, lse_used=f64(lse))
    first = x.grad.clone(), w.grad.clone()
    vt.head_loss(x, w, t, 2, 96, **p.how).mean().backward()
    even = torch.full_like(g, 1 / 50)
    second = vt.head_xent_grad(x.detach(), w.detach(), t, lse, even, 2, 96, **p.how)
    assert torch.equal(x.grad, first[0] + second[0]) and torch.equal(w.grad, first[1] + second[1])


@gpu
def test_work_arrays_past_32_bits():
    """d of 20001 rows by 131000 entries is 5.2 GB in one piece: offsets in
    bytes and in elements pass 32 bits."""
    print("[gpu] large d", flush=True)
    m, rows, vocab, hidden = 20001, 131072, 131000, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, hidden, generator=g, device=DEV).bfloat16()
    w = (torch.randn(rows, hidden, generator=g, device=DEV) * 0.1).bfloat16()
    labels = torch.randint(0, vocab, (m,), generator=g, device=DEV)
    grad = 0.5 + torch.rand(m, generator=g, device=DEV)
    loss, lse, dx, dw = vt.head_xent_step(x, w, labels, grad, 8, rows // 8, vocab=vocab, workspace_limit=0,
                                          dw=torch.empty(rows, hidden, device=DEV))
    wd, want_w, at = w[:vocab].double(), torch.zeros(rows, hidden, dtype=torch.float64, device=DEV), 0
    for rx, rt, rg, rl, rd in zip(*(v.split(2500) for v in (x, labels, grad, loss, dx))):
        logp = torch.log_softmax(rx.double() @ wd.t(), dim=1)
        here = torch.arange(len(rt), device=DEV)
        # fp32 sums of 64 products and of 131000 exponentials, joined by tiles
        assert ((rl.double() + logp[here, rt]).abs() <= 1e-5).all()
        d = logp.exp_()
        d[here, rt] -= 1.0
        d *= rg[:, None].double()
        want = d @ wd
        # one rounding of the result; the probabilities' own are 1/362 of the label's
        assert float((rd.double() - want).norm() / want.norm()) <= 1.1 * float(
            (want.bfloat16().double() - want).norm() / want.norm())
        want_w[:vocab] += d.t() @ rx.double()
    assert float((dw.double() - want_w).norm() / want_w.norm()) <= 0.1 * 2.0 ** -8
    assert not dw[vocab:].any()
    del logp, d, want_w, dw
    torch.cuda.empty_cache()
