"""Arguments of the training operators' Python calls that are refused before
anything is asked of the library (CPU)."""

from __future__ import annotations

import pytest
import torch

from tp_vocab_logits_amd import _lib
from tp_vocab_logits_amd import vocab_train as vt


@pytest.mark.parametrize("limit", [-1, -(1 << 40)])
def test_a_negative_workspace_limit_is_refused(limit):
    shape = (1, 64, 16, 4, 60, _lib.HG_BF16, 8)
    assert vt._xent_bytes(shape, _lib.HG_XENT_STEP, 0) > 0
    with pytest.raises(ValueError):
        vt._xent_bytes(shape, _lib.HG_XENT_STEP, limit)


@pytest.mark.parametrize("blocks", [[None, None], ["w", "w"], [torch.tensor(1.0)] * 2, [torch.zeros(64, 16).bfloat16(), None],
                                    [torch.zeros(64).bfloat16()] * 2, [torch.zeros(64, 16).numpy()] * 2])
def test_blocks_that_are_no_matrices_are_refused(blocks):
    x, t = torch.zeros(3, 16).bfloat16(), torch.zeros(3).long()
    with pytest.raises(ValueError):
        vt.head_xent(x, blocks, t, 2, 64)
    with pytest.raises(ValueError):
        vt.embed(t, blocks, 2, 64)


@pytest.mark.parametrize("w", [None, 3, 1.5])
def test_a_matrix_that_is_neither_a_tensor_nor_blocks_is_refused(w):
    with pytest.raises(ValueError):
        vt.embed(torch.zeros(3).long(), w, 1, 64)


@pytest.mark.parametrize("kind", [tuple, iter, torch.nn.ParameterList])
def test_blocks_come_in_any_iterable(kind):
    blocks = [torch.zeros(64, 16).bfloat16() for _ in range(2)]
    assert vt._matrix(kind(blocks), 2, 64, (torch.bfloat16,))[1] == 16
