"""A tied vocabulary matrix trained at both of its ends.

The smallest language model there is: a token's embedding, plus one linear map
of it, predicts the next token through the same matrix. Per step:

    h      = embed(tokens, W, scale=sqrt(H))        lookup with scaling
    x      = norm(h + h @ A)                        torch
    loss   = cross entropy of x @ W.T, no logits    head_xent_step: loss, dx, dW
    dW    += embed_grad(tokens, dh, scale=sqrt(H))  the lookup's part of the tied gradient
    W, A  -= lr * gradient                          torch

Text is synthetic: a random permutation of the vocabulary is followed nine times
out of ten, so a model that learns gets well below log(vocab).

    python examples/tied_vocab_training.py [--steps 60]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tp_vocab_logits_amd import embed, embed_grad, head_xent, head_xent_step  # noqa: E402


def batches(vocab: int, rows: int, seed: int, device):
    """Endless (tokens, labels): labels follow a fixed permutation, or are noise;
    a tenth of the rows is left out, as a prompt's would be."""
    g = torch.Generator().manual_seed(seed)
    follows = torch.randperm(vocab, generator=g)
    while True:
        tokens = torch.randint(0, vocab, (rows,), generator=g)
        noise = torch.randint(0, vocab, (rows,), generator=g)
        labels = torch.where(torch.rand(rows, generator=g) < 0.9, follows[tokens], noise)
        labels[torch.rand(rows, generator=g) < 0.1] = -100
        yield tokens.to(device), labels.to(device)


def train(steps: int, tp: int = 4, shard: int = 256, vocab: int = 1000, hidden: int = 256, rows: int = 4096,
          lr: float = 0.5, seed: int = 0, device="cuda:0", tell=print) -> list[float]:
    """The mean loss of every step."""
    g = torch.Generator().manual_seed(seed)
    w32 = (torch.randn(tp * shard, hidden, generator=g) * 0.02).to(device)  # master weights
    a = torch.zeros(hidden, hidden, device=device, requires_grad=True)
    scale = math.sqrt(hidden)
    data, losses = batches(vocab, rows, seed + 1, device), []
    for step in range(steps):
        tokens, labels = next(data)
        w = w32.bfloat16()
        h = embed(tokens, w, tp, shard, scale=scale).requires_grad_()
        hf = h.float()
        x = torch.nn.functional.rms_norm(hf + hf @ a, (hidden,)).bfloat16()
        count = (labels != -100).sum().clamp(min=1)
        grad = torch.ones(rows, device=device) / count
        dw = torch.empty(tp * shard, hidden, device=device)  # fp32: both ends add up in it
        loss, _, dx, dw = head_xent_step(x.detach(), w, labels, grad, tp, shard, vocab=vocab, dw=dw)
        a.grad = None
        x.backward(dx)
        embed_grad(tokens, h.grad, tp, shard, scale=scale, dw=dw, accumulate=True)
        with torch.no_grad():
            norm = dw.norm().clamp(min=1e-12)
            w32 -= lr * dw * (1.0 / norm).clamp(max=4.0)
            a -= lr * a.grad
        losses.append(float(loss.sum() / count))
        if step % 10 == 0 or step == steps - 1:
            tell(f"step {step:3d}  loss {losses[-1]:.4f}  (uniform {math.log(vocab):.4f})")
    # scoring: the log-probability of the right next token
    tokens, labels = next(data)
    w = w32.bfloat16()
    with torch.no_grad():
        hf = embed(tokens, w, tp, shard, scale=scale).float()
        x = torch.nn.functional.rms_norm(hf + hf @ a, (hidden,)).bfloat16()
    nll, _ = head_xent(x, w, labels, tp, shard, vocab=vocab)
    tell(f"held out: {float(nll.sum() / (labels != -100).sum()):.4f} nats per token")
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps)
