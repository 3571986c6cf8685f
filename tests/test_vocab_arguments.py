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
