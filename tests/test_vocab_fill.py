"""The zeros that an embedding gradient writes beside its sort: a grid that any
gradient's size fits (CPU), and a gradient larger than one store per thread
reaches (GPU)."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from tp_vocab_logits_amd import build
from tp_vocab_logits_amd import vocab_train as vt

DEV = "cuda:0"
MOST_LANES = 1 << 32  # a launch has fewer


@pytest.fixture(scope="module")
def fill_groups(tmp_path_factory):
    d = tmp_path_factory.mktemp("fill")
    src, so = d / "fill.cpp", d / "fill.so"
    src.write_text('#include "hg_fill.h"\nextern "C" int groups(long long v) { return hg::fill_groups(v); }\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o",
                    str(so)], check=True)
    fn = ctypes.CDLL(str(so)).groups
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_longlong]
    return fn


def test_a_fill_of_any_size_fits_a_launch(fill_groups):
    assert [fill_groups(v) for v in (-5, 0, 1, 1024, 1025, 1 << 20)] == [0, 0, 1, 1, 2, 1024]
    largest = (1 << 29) * (1 << 20) * 4 // 16  # rows x hidden that hg_embed_grad takes, in fp32
    for bits in range(20, 48):
        for vecs in (1 << bits, (1 << bits) + 1, 3 << bits):
            groups = fill_groups(min(vecs, largest))
            assert 0 < groups * 1024 < MOST_LANES // 2


@pytest.mark.gpu
@pytest.mark.parametrize("n", [300, 5000])
def test_a_gradient_of_more_zeros_than_threads(n):
    """5 GB: the fill beside a sort of one launch goes round; beside six it does not."""
    print(f"[gpu] large fill {n=}", flush=True)
    rows, hidden = 5 * (1 << 22) + 3, 64
    g = torch.Generator(device=DEV).manual_seed(n)
    tokens = torch.randint(-1, rows, (n,), generator=g, device=DEV)
    tokens[:3] = torch.tensor([0, rows - 1, rows], device=DEV)
    dy = torch.randn(n, hidden, generator=g, device=DEV)
    dw = torch.full((rows, hidden), float("nan"), device=DEV)
    vt.embed_grad(tokens, dy, 1, rows, dw=dw)
    kept = (tokens >= 0) & (tokens < rows)
    named, where = torch.unique(tokens[kept], return_inverse=True)
    want = torch.zeros(len(named), hidden, dtype=torch.float64, device=DEV).index_add_(0, where, dy[kept].double())
    assert ((dw[named].double() - want).abs() <= 1e-6 * (1 + want.abs())).all()
    dw[named] = 0
    assert int(torch.count_nonzero(dw)) == 0
    del dw
    torch.cuda.empty_cache()
