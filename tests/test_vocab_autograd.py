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
