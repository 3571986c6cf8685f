"""The differentiable forms as a training program uses them: results changed in
place, gradients that add up, arguments that reach the backward pass (GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from test_vocab_train import DEV, Problem, f64
from tp_vocab_logits_amd import vocab_train as vt

gpu = pytest.mark.gpu
ARGS = (2, 96)


def leaves(p, frozen=()):
    x, w, t, g = p.on_gpu()
    return x.requires_grad_("x" not in frozen), w.requires_grad_("w" not in frozen), t, g


@gpu
def test_the_loss_can_be_changed_in_place():
    """As torch's own cross entropy can: weighted rows, a mask."""
    print("[gpu] loss in place", flush=True)
    p = Problem(*ARGS, 64, 50, 150, left_out=0.2)
    x, w, t, g = leaves(p)
    loss = vt.head_loss(x, w, t, *ARGS, **p.how)
    plain = loss.detach().clone()
    loss *= g
    assert torch.equal(loss, plain * g)
    loss.sum().backward()
    lse = vt.head_xent(x.detach(), w.detach(), t, *ARGS, **p.how)[1]
    p.check_grads(x.grad, w.grad, lse_used=f64(lse))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tp,shard,hidden,m", [(2, 96, 64, 50), (2, 8480, 520, 300), (1, 256, 1024, 2500)])
def test_a_frozen_side_gets_no_gradient(tp, shard, hidden, m, dtype):
    """Small and big tiles, and sums that are split: the other side's gradient
    is the same bits."""
    print(f"[gpu] frozen {tp=} {shard=} {hidden=} {m=} {dtype}", flush=True)
    p = Problem(tp, shard, hidden, m, tp * shard - 7, dtype, left_out=0.1, scale=0.7, z_weight=0.01)
    got = {}
    for frozen in ((), ("x",), ("w",)):
        x, w, t, g = leaves(p, frozen)
        (vt.head_loss(x, w, t, tp, shard, **p.how) * g).sum().backward()
        got[frozen] = x.grad, w.grad
    assert got["x",][0] is None and torch.equal(got["x",][1], got[()][1])
    assert got["w",][1] is None and torch.equal(got["w",][0], got[()][0])


@gpu
@pytest.mark.parametrize("frozen", [(), ("x",), ("w",)])
def test_no_rows(frozen):
    print(f"[gpu] no rows {frozen}", flush=True)
    x, w, t, _ = leaves(Problem(*ARGS, 64, 0, 150), frozen)
    vt.head_loss(x, w, t, *ARGS, vocab=150).sum().backward()
    assert x.grad is None if "x" in frozen else x.grad.shape == (0, 64)
    assert w.grad is None if "w" in frozen else not w.grad.any()


@gpu
def test_a_frozen_matrix_costs_no_gradient_of_it():
    """The backward pass of a frozen head allocates nothing of the matrix's size."""
    print("[gpu] frozen memory", flush=True)
    p = Problem(2, 8192, 1024, 64)
    x, w, t, _ = leaves(p, ("w",))
    loss = vt.head_loss(x, w, t, 2, 8192, **p.how).sum()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    loss.backward()
    assert torch.cuda.max_memory_allocated() - before < w.numel() * w.element_size()


@gpu
def test_the_backward_pass_keeps_within_its_workspace_limit():
    print("[gpu] workspace limit", flush=True)
    p = Problem(2, 16384, 64, 2000, left_out=0.1)
    got, took = [], []
    for limit in (vt.WORKSPACE_LIMIT, 16 << 20):
        x, w, t, g = leaves(p)
        loss = (vt.head_loss(x, w, t, 2, 16384, workspace_limit=limit, **p.how) * g).sum()
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        loss.backward()
        took.append(torch.cuda.max_memory_allocated() - before)
        got.append((x.grad, w.grad))
    assert took[0] > 2 * 2000 * 32768 and took[1] < 32 << 20
    lse = f64(vt.head_xent(x.detach(), w.detach(), t, 2, 16384, **p.how)[1])
    for dx, dw in got:
        p.check_grads(dx, dw, lse_used=lse)


@gpu
def test_both_passes_replay_in_a_graph():
    """Captured with no other autograd graph of the same leaves alive; every
    replay against the eager result of the same inputs."""
    print("[gpu] autograd in a graph", flush=True)
    p = Problem(2, 320, 136, 70, 601, left_out=0.1, z_weight=0.01)
    x, w, t, g = leaves(p)
    tokens = torch.randint(0, 640, (70,), generator=torch.Generator().manual_seed(1)).to(DEV)

    def both(x, w):
        loss = vt.head_loss(x + vt.embedding(tokens, w, 2, 320, 3.0), w, t, 2, 320, **p.how)
        return (loss.detach(), *torch.autograd.grad((loss * g).sum(), (x, w)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(x, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x, w)
    for k in range(4):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)))
        want = both(x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k
