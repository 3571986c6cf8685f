"""What the calls that write into their arguments mean to autograd: a tensor that a backward pass needs and that was
overwritten is noticed there, and one whose gradient would leave the adapters out is refused."""

from __future__ import annotations

import pytest
import torch

from tp_vocab_logits_amd import adapt, beam_reorder

DEV = "cuda:0"
gpu = pytest.mark.gpu


def low(device, m=5, n=2, rank=8, hidden=16, v=24):
    g = torch.Generator().manual_seed(1)
    x, a, b = (torch.randn(s, generator=g).bfloat16().to(device) for s in ((m, hidden), (n, rank, hidden), (n, v, rank)))
    return x, a, b, torch.zeros(m, dtype=torch.int64, device=device), 1, v


def test_out_of_a_graph_is_refused():
    y = torch.zeros(5, 24, dtype=torch.bfloat16)
    for out in (y.clone().requires_grad_(), y.clone().requires_grad_() * 1, (y.clone().requires_grad_() * 1)[:]):
        for source in (y, out):
            with pytest.raises(ValueError, match="adapted"):
                adapt(source, *low("cpu"), out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # as torch's own in-place calls: then it is allowed
        adapt(y, *low("cpu"), out=y.clone().requires_grad_())


@gpu
@pytest.mark.parametrize("m", [5, 90])
def test_an_output_that_was_saved_is_noticed(m):
    leaf = torch.ones(m, 24, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    for out in (torch.ones(m, 24, dtype=torch.bfloat16, device=DEV), leaf * 2):
        z = (out * leaf).sum()
        with torch.no_grad():
            before = out._version
            adapt(out, *low(DEV, m), out=out)
        assert out._version == before + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
    y = torch.ones(m, 24, dtype=torch.bfloat16, device=DEV)
    z = (y * leaf).sum()
    adapt(y, *low(DEV, m), out=torch.empty_like(y))  # y is read only
    adapt(y, *low(DEV, m))
    z.backward()
    assert torch.equal(leaf.grad, y)


@gpu
def test_states_that_were_saved_are_noticed():
    p = torch.tensor([[1, 0]], device=DEV)
    leaf = torch.ones(2, 3, device=DEV, requires_grad=True)
    cache, other = torch.ones(2, 2, 3, device=DEV), torch.ones(2, 3, device=DEV)
    z, w = (cache[:, 1] * leaf).sum(), (other * leaf).sum()
    versions = cache._version, other._version
    beam_reorder([cache[:, 0], other], p)
    assert (cache._version, other._version) == (versions[0] + 1, versions[1] + 1)  # (a view shares its base's)
    for t in (z, w):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            t.backward()


@gpu
def test_under_inference_and_captured():
    args, p = low(DEV), torch.tensor([[1, 0]], device=DEV)
    y = torch.ones(5, 24, dtype=torch.bfloat16, device=DEV)
    want = adapt(y, *args)
    with torch.inference_mode():
        t, s = torch.ones(5, 24, dtype=torch.bfloat16, device=DEV), torch.arange(6.0, device=DEV).view(2, 3)
        assert torch.equal(adapt(t, *args, out=t), want)
        beam_reorder(s, p)
        assert s.tolist() == [[3, 4, 5], [0, 1, 2]]
    t, s = torch.ones_like(y), torch.arange(6.0, device=DEV).view(2, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adapt(t, *args, out=t)
        beam_reorder(s, p)
    for k in range(3):
        t.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t, want)
        assert s.tolist() == ([[0, 1, 2], [3, 4, 5]] if k % 2 else [[3, 4, 5], [0, 1, 2]])
