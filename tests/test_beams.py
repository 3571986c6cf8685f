"""Beam search's operators: the oracle against torch in float64, argument checks
and refusals (CPU); the kernels against the oracle (GPU)."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import beams as ob
from tp_vocab_logits_amd import _lib, beam_reorder, beam_select
from tp_vocab_logits_amd import beams as tb
from tp_vocab_logits_amd._lib import HgError

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
gpu = pytest.mark.gpu


def note(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)


def rand(shape, seed, dtype="fp32", sigma=3.0) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(DT[dtype])


# -- the oracle ---------------------------------------------------------------


def test_oracle_selection_is_torchs():
    z, s = rand((3, 4, 11), 1).double(), rand((3, 4), 2).double()
    c = (torch.log_softmax(0.7 * z, dim=2) + s[..., None]).reshape(3, -1)
    want, at = c.topk(9, dim=1)
    out, parents, tokens = ob.beam_select(z.numpy(), s.numpy(), 9, scale=0.7)
    np.testing.assert_allclose(out, want.numpy(), rtol=1e-13)
    assert (parents * 11 + tokens == at.numpy()).all()


def test_oracle_special_rows():
    inf, nan = np.inf, np.nan
    z = np.array([[[0.0, nan, 0.0, -inf], [inf, 5.0, inf, nan], [-inf] * 4, [1.0] * 4]])
    out, parents, tokens = ob.beam_select(z, np.array([[0.0, 0.0, 0.0, -inf]]), 6)
    assert parents.tolist() == [[0, 0, 1, 1, -1, -1]] and tokens.tolist() == [[0, 2, 0, 2, -1, -1]]
    np.testing.assert_allclose(out[0, :4], -np.log(2.0))
    out, parents, tokens = ob.beam_select(z, np.array([[-9.0, nan, inf, -1.0]]), 3, np.array([[0, 0, 0, 1]]), 3)
    assert parents.tolist() == [[3, 0, 0]] and tokens.tolist() == [[3, 0, 2]] and out[0, 0] == -1.0


def test_oracle_reorder_is_an_index():
    t = rand((6, 2, 5), 3).numpy()
    p = np.array([[1, 1, 0], [2, -1, 7]])
    want = t[[1, 1, 0, 5, 4, 5]]
    assert (ob.beam_reorder(t, p) == want).all()
    got = ob.beam_reorder(t, p, np.array([2, 9]), 2)
    assert (got[:3, :, :2] == want[:3, :, :2]).all() and (got[:3, :, 2:] == t[:3, :, 2:]).all()
    assert (got[3:] == want[3:]).all()


# -- refusals -----------------------------------------------------------------


def test_selection_checks_its_arguments():
    z, s = torch.zeros(6, 10), torch.zeros(2, 3)
    for bad in (dict(scores=torch.zeros(6)), dict(scores=s.double()), dict(scores=s.t()), dict(logits=z[:5]),
                dict(logits=z.double()), dict(logits=z.t()), dict(logits=None), dict(logits=[]),
                dict(logits=[z, z.bfloat16()]), dict(logits=[z, z[:, :4]]), dict(logits=torch.zeros(65, 6, 1)),
                dict(finished=torch.zeros(2, 3)), dict(finished=torch.zeros(3, 2, dtype=torch.bool))):
        with pytest.raises(ValueError):
            beam_select(**{"logits": z, "scores": s, "keep": 4, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        beam_select(z, s, 4)


def test_library_checks_the_selection():
    lib = _lib.lib()
    n = ctypes.c_size_t()
    good = dict(requests=2, beams=3, keep=4, tp=2, shard=10, vocab=17, dtype=_lib.HG_BF16, pad=0, scale=1.0)
    assert lib.hg_beam_workspace(_lib.BeamShape(**good), n) == 0 and n.value > 0
    assert lib.hg_beam_workspace(_lib.BeamShape(**good), None) == _lib.HG_EINVAL
    assert lib.hg_beam_workspace(None, n) == _lib.HG_EINVAL
    for bad in (dict(requests=-1), dict(beams=0), dict(beams=65), dict(keep=0), dict(keep=65), dict(tp=0),
                dict(tp=65), dict(shard=0), dict(vocab=0), dict(vocab=21), dict(dtype=3), dict(pad=-1), dict(pad=17),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
                dict(shard=1 << 20, vocab=(1 << 20) + 1), dict(requests=1 << 30), dict(requests=(1 << 23) + 1, beams=1)):
        assert lib.hg_beam_workspace(_lib.BeamShape(**{**good, **bad}), n) == _lib.HG_EINVAL, bad
    shape = _lib.BeamShape(**good)
    ptrs = _lib.pointer_array([1 << 20, 2 << 20])
    args = [3 << 20, 0, 4 << 20, 5 << 20, 6 << 20, 7 << 20, 1 << 19]

    def call(logits=ptrs, s=shape, **at):
        a = list(args)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.hg_beam_select(s, logits, *a, None)

    assert call(a6=16) == _lib.HG_ESIZE
    assert call(a0=None) == call(a2=None) == call(a3=None) == call(a4=None) == call(a5=None) == _lib.HG_EINVAL
    assert call(a0=(3 << 20) + 2) == call(a2=(4 << 20) + 2) == call(a3=(5 << 20) + 4) == _lib.HG_EINVAL
    assert call(a5=(7 << 20) + 16) == call(logits=None) == _lib.HG_EINVAL
    assert call(logits=_lib.pointer_array([1 << 20, 0])) == _lib.HG_EINVAL
    assert call(logits=_lib.pointer_array([1 << 20, (2 << 20) + 1])) == _lib.HG_EINVAL
    assert call(a2=3 << 20) == call(a3=4 << 20) == call(a5=1 << 20) == call(a1=7 << 20) == _lib.HG_EINVAL  # overlaps
    assert call(s=_lib.BeamShape(**{**good, "requests": 0}), a0=None) == _lib.HG_OK


def state(ptr, row, outer_stride, step, outer, steps):
    return _lib.BeamState(ptr, row, outer_stride, step, outer, steps)


def test_library_checks_the_reordering():
    lib = _lib.lib()
    mb = 1 << 20

    def call(*states, requests=2, beams=2, parents=9 * mb, pb=8, lengths=None, lb=8):
        a = (_lib.BeamState * max(1, len(states)))(*states)
        return lib.hg_beam_reorder(requests, beams, len(states), a, parents, pb, lengths, lb, None)

    one = state(mb, 100, 0, 10, 1, 10)
    bad = _lib.HG_EINVAL
    assert call() == call(one, requests=0) == _lib.HG_OK
    assert call(state(0, 100, 0, 10, 1, 0)) == call(state(0, 0, 0, 0, 0, 5)) == _lib.HG_OK  # empty states
    assert call(one, requests=-1) == call(one, beams=0) == call(one, beams=65) == call(one, pb=2) == bad
    assert call(one, parents=None) == call(one, parents=9 * mb + 4) == call(one, lengths=mb * 8 + 2, lb=4) == bad
    assert call(one, lengths=mb * 8, lb=3) == call(state(0, 100, 0, 10, 1, 10)) == bad
    assert call(state(mb, 99, 0, 10, 1, 10)) == call(state(mb, 0, 0, 10, 1, 10)) == bad  # rows into each other
    assert call(state(mb, 100, 99, 10, 2, 10)) == call(state(mb, 100, 150, 10, 2, 10)) == bad
    assert call(state(mb, -100, 0, 10, 1, 10)) == call(state(mb, 100, 0, -1, 1, 10)) == bad
    assert call(state(mb, 100, 0, 10, -1, 10)) == call(state(mb, 100, 0, 10, 1, -1)) == bad
    assert call(state(mb, 1 << 60, 0, 10, 1, 10)) == call(state(mb, 100, 0, 1 << 50, 1, 10)) == bad
    assert call(one, one) == call(one, state(mb + 399, 100, 0, 10, 1, 10)) == bad  # into each other
    assert call(one, state(mb + 50, 100, 0, 10, 1, 5)) == call(one, parents=mb + 392) == bad
    assert call(one, lengths=mb + 384, lb=8) == bad
    # states may lie between each other's runs, not share a byte (views that
    # touch are tested where there is a cache to move)
    k, v = state(mb, 200, 400 * 4, 10, 3, 10), state(mb + 100, 200, 400 * 4, 10, 3, 10)
    assert call(k, state(mb + 99, 200, 400 * 4, 10, 3, 10)) == bad
    assert call(k, state(mb + 200, 200, 400 * 4, 10, 3, 10)) == bad  # its rows from the second on
    assert call(k, v, k) == bad
    # more work than a launch covers, before anything is launched
    assert call(state(mb, 1 << 40, 0, 1 << 30, 1, 1 << 10), requests=64, beams=1, parents=1 << 60) == bad


@pytest.mark.parametrize("shape,strides,dim,want", [
    ((6, 5), (5, 1), 1, (20, 0, 4, 1, 5)),
    ((6, 5), (5, 1), None, (20, 0, 20, 1, 1)),
    ((6,), (1,), None, (4, 0, 4, 1, 1)),
    ((6, 2, 3, 4), (24, 12, 4, 1), 2, (96, 48, 16, 2, 3)),
    ((6, 2, 3, 4), (24, 12, 4, 1), 1, (96, 0, 48, 1, 2)),
    ((6, 2, 3, 4), (24, 12, 4, 1), None, (96, 0, 96, 1, 1)),
    ((6, 2, 3, 4), (12, 72, 4, 1), 2, (48, 288, 16, 2, 3)),  # heads outside of the rows
    ((6, 2, 3, 4), (12, 72, 4, 1), None, (48, 288, 48, 2, 1)),
    ((6, 1, 3, 1), (3, 7, 1, 9), 2, (12, 0, 4, 1, 3)),
    ((6, 2, 2, 3, 4), (48, 24, 12, 4, 1), 3, (192, 48, 16, 4, 3)),
    ((6, 0, 3), (3, 3, 1), 2, (0, 0, 0, 0, 0)),
])
def test_geometry_of_states(shape, strides, dim, want):
    assert tb._geometry(shape, strides, 4, dim) == want


@pytest.mark.parametrize("shape,strides,dim", [
    ((6, 5), (10, 2), 1), ((6, 5), (5, 1), 0), ((6, 5), (5, 1), 2), ((), (), None), ((6, 3, 4), (24, 8, 1), 1),
    ((6, 2, 2, 3), (100, 50, 9, 1), 3), ((6, 2, 2, 3), (100, 50, 9, 1), None)])
def test_states_with_gaps_are_refused(shape, strides, dim):
    with pytest.raises(ValueError):
        tb._geometry(shape, strides, 4, dim)


def test_reordering_checks_its_arguments():
    t, p = torch.zeros(6, 4), torch.zeros(2, 3, dtype=torch.int64)
    for bad in (dict(parents=p.float()), dict(parents=p.t()), dict(parents=p[0]), dict(states=torch.zeros(5, 4)),
                dict(states=[t, None]), dict(states=torch.zeros(6, 4, requires_grad=True)),
                dict(lengths=torch.zeros(2, dtype=torch.int64)), dict(lengths=torch.zeros(2), time_dim=1),
                dict(lengths=torch.zeros(3, dtype=torch.int64), time_dim=1), dict(time_dim=2), dict(time_dim=0),
                dict(parents=torch.zeros(1, 65, dtype=torch.int64), states=torch.zeros(65, 1))):
        with pytest.raises(ValueError):
            beam_reorder(**{"states": t, "parents": p, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        beam_reorder(t, p)


# -- selection on the GPU -----------------------------------------------------


def blocks_of(z, tp, vocab):
    """[rows, vocab] as [tp, rows, shard], NaN in the padding."""
    rows, shard = z.shape[0], -(-vocab // tp)
    full = torch.full((rows, tp * shard), math.nan, dtype=z.dtype)
    full[:, :vocab] = z
    return full.view(rows, tp, shard).transpose(0, 1).contiguous()


def compare(got, z, s, keep, finished=None, pad=0, scale=1.0):
    """Parents and tokens are the oracle's; a score is rounded once (half a step of
    fp32) from sums that are right to 6e-11 and a few steps of float64."""
    requests, beams = s.shape
    want = ob.beam_select(z.double().numpy().reshape(requests, beams, -1), s.double().numpy(), keep,
                          None if finished is None else finished.numpy(), pad, float(torch.tensor(scale)))
    out, parents, tokens = (t.cpu().numpy() for t in got)
    np.testing.assert_array_equal(parents, want[1])
    np.testing.assert_array_equal(tokens, want[2])
    with np.errstate(over="ignore"):
        bound = np.abs(want[0]) * (2.0 ** -24 + 1e-14) + 1e-9
    real = want[1] >= 0
    assert (out[~real] == -np.inf).all()
    fits = real & (np.abs(want[0]) < 3.4e38)
    assert (np.abs(out[fits] - want[0][fits]) <= bound[fits]).all()


def select(z, s, keep, tp=0, vocab=None, finished=None, **how):
    d = blocks_of(z, tp, z.shape[1]) if tp else z
    vocab = z.shape[1] if vocab is None else vocab
    got = beam_select(d.to(DEV), s.to(DEV), keep, vocab=vocab,
                      finished=None if finished is None else finished.to(DEV), **how)
    return got


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("requests,beams,keep,vocab,tp", [
    (1, 1, 1, 1, 0), (1, 1, 5, 3, 0), (1, 4, 8, 163840, 0), (3, 2, 4, 1000, 0), (2, 5, 10, 4091, 0),
    (7, 3, 6, 2049, 3), (1, 2, 64, 5000, 4), (2, 64, 64, 301, 0), (5, 8, 16, 31999, 4), (1, 33, 40, 777, 64),
    (40, 4, 8, 20480, 8), (1, 1, 3, 70001, 7)])
def test_selection(dtype, requests, beams, keep, vocab, tp):
    note(f"select {dtype} {requests} {beams} {keep} {vocab} {tp}")
    z, s = rand((requests * beams, vocab), vocab + keep, dtype), rand((requests, beams), 5) - 10
    compare(select(z, s, keep, tp), z, s, keep)


@gpu
@pytest.mark.parametrize("dtype,vecs", [("bf16", 1), ("bf16", 2), ("bf16", 4), ("fp32", 2), ("fp32", 4)])
def test_selection_of_every_part_size(dtype, vecs):
    # the part grows while rows x parts are more than 2048: 9, 5 and 3 parts of bf16, 17, 9 and 5 of fp32
    rows = {1: 100, 2: 300 if dtype == "bf16" else 200, 4: 2000}[vecs]
    vocab = 8 * 2048 + 5
    note(f"select parts {dtype} {vecs}")
    z, s = rand((rows, vocab), vecs, dtype), rand((rows // 4, 4), 6)
    compare(select(z, s, 8), z, s, 8)


@gpu
@pytest.mark.parametrize("offset", [1, 3, 5, 7])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_start_anywhere(dtype, offset):
    note(f"select offset {dtype} {offset}")
    z, s = rand((6, 4093), offset, dtype), rand((2, 3), 7)
    room = torch.full((6 * 4093 + 16,), math.nan, dtype=DT[dtype], device=DEV)
    part = room[offset:offset + z.numel()].view(6, 4093)
    part.copy_(z)
    compare(beam_select(part, s.to(DEV), 6), z, s, 6)


def special_rows(kind, dtype, vocab):
    t = DT[dtype]
    z = rand((8, vocab), 11, dtype)
    if kind == "constant":
        z[:] = 0.25
    elif kind == "few values":
        z = (z.float() / 3).round().to(t)
    elif kind == "rising":
        z[:] = (torch.arange(vocab) / vocab * 8 - 4).to(t)
    elif kind == "falling":
        z[:] = (4 - torch.arange(vocab) / vocab * 8).to(t)
    elif kind == "zeros of both signs":
        z[:] = 0.0
        z[:, 1::2] = -0.0
        z[:, ::7] = -1.0
    elif kind == "masked":
        z[:, torch.arange(vocab) % 3 != 1] = -math.inf
        z[2] = -math.inf
        z[3, 5:] = -math.inf
    elif kind == "lowest":
        z[:, torch.arange(vocab) % 3 != 1] = torch.finfo(t).min
        z[2] = torch.finfo(t).min
        z[3, 2:] = torch.finfo(t).min
    elif kind == "nan":
        z[:, ::5] = math.nan
        z[1] = math.nan
        z[2, : vocab // 2] = math.nan
        z[4, 1:] = math.nan
    elif kind == "infinite":
        z[0, 3] = math.inf
        z[1, ::17] = math.inf
        z[2] = math.inf
        z[3, 9] = math.nan
        z[3, vocab - 1] = math.inf
        z[5] = -math.inf
        z[5, 2] = math.inf
    elif kind == "one part":  # the best of a row follow one another
        z[:, vocab // 2: vocab // 2 + 300] += 40.0
    return z


KINDS = ["constant", "few values", "rising", "falling", "zeros of both signs", "masked", "lowest", "nan", "infinite",
         "one part"]


@gpu
@pytest.mark.parametrize("keep", [3, 16, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_special_rows(kind, dtype, keep):
    note(f"select {kind} {dtype} {keep}")
    vocab = 40003
    z, s = special_rows(kind, dtype, vocab), torch.tensor([[0.0, -1.5, -2.0, -0.25], [-3.0, -3.0, -3.5, -4.0]])
    compare(select(z, s, keep), z, s, keep)
    compare(select(z, s, keep, tp=3), z, s, keep)


@gpu
def test_many_to_keep_of_rows_in_order():
    # every part holds more of the best than the join's LDS has room for
    vocab = 1 << 18
    z = (torch.arange(vocab) / vocab * 8 - 4).repeat(64, 1)
    s = rand((1, 64), 8)
    note("select 64 of 64 rising rows")
    compare(select(z, s, 64), z, s, 64)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_longest_rows(dtype):
    z, s = rand((2, 1 << 20), 12, dtype), rand((1, 2), 9)
    note(f"select 2^20 {dtype}")
    compare(select(z, s, 9), z, s, 9)
    compare(select(z, s, 64, tp=64), z, s, 64)


@gpu
def test_beams_that_are_not_there():
    z = rand((12, 5000), 13, "bf16")
    s = torch.tensor([[-1.0, -math.inf, -2.0, math.nan], [-math.inf] * 4, [math.inf, -3.0, -3.0, -math.inf]])
    z[1], z[3], z[4:8], z[8] = math.nan, math.inf, math.nan, math.nan  # never read
    note("select dead beams")
    compare(select(z, s, 8), z, s, 8)
    compare(select(z[:, :3].contiguous(), s, 8), z[:, :3], s, 8)


@gpu
@pytest.mark.parametrize("pad", [0, 2, 4999])
def test_finished_beams(pad):
    z, s = rand((12, 5000), 14, "fp16"), rand((3, 4), 10) - 5
    finished = torch.tensor([[1, 0, 0, 1], [1, 1, 1, 1], [0, 0, 0, 0]], dtype=torch.bool)
    s[0, 3] = -math.inf
    s[1] = -7.0  # ties among finished beams
    z[0], z[4:8] = math.nan, math.nan
    z[1, pad] = -math.inf
    note(f"select finished {pad}")
    compare(select(z, s, 6, finished=finished, pad=pad), z, s, 6, finished, pad)


@gpu
@pytest.mark.parametrize("scale", [1e-3, 0.7, 12.5, 1e30])
def test_scaled_logits(scale):
    z, s = rand((6, 3001), 15), rand((2, 3), 11)
    note(f"select scale {scale}")
    compare(select(z, s, 5, scale=scale), z, s, 5, scale=scale)


@gpu
def test_order_over_beams_is_the_64_bit_one():
    """Two beams whose candidates differ by 3e-8 of a sum of 20000 terms: an error of 1e-7 in a row's sum would
    swap them."""
    vocab = 20000
    z = rand((2, vocab), 16, "bf16").float()
    z[1] = z[0]
    z[:, 0] = 20.0
    for step in (3e-8, -3e-8):
        s = torch.tensor([[0.0, 0.0]])
        z[1, 0] = 20.0
        lse = torch.logsumexp(z[0, 1:].double(), 0)
        # the second row's other logits are shifted so that its first candidate moves by `step`
        p = (torch.exp(lse) / (torch.exp(lse) + math.exp(20.0))).item()
        z[1, 1:] = (z[0, 1:].double() - step / p).float()
        c = ob.candidates(z.double().numpy()[None], s.double().numpy())[0, :, 0]
        assert 1e-9 < abs(c[1] - c[0]) < 1e-6
        note(f"select near ties {step}")
        compare(select(z, s, 2), z, s, 2)


@gpu
def test_identical_beams_tie_by_place():
    z = rand((1, 30000), 17, "bf16").repeat(4, 1)
    s = torch.full((1, 4), -2.0)
    note("select identical beams")
    got = select(z, s, 8)
    assert got[1].tolist() == [[0, 1, 2, 3, 0, 1, 2, 3]] or len(set(got[0][0, :4].tolist())) == 1
    compare(got, z, s, 8)


@gpu
def test_selection_past_32_bit_offsets():
    rows, vocab = 14000, 163840  # 4.6 GB
    note("select 4.6 GB")
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device=DEV)
    tail = rand((8, vocab), 18, "bf16")
    z[-8:] = tail.to(DEV)
    s = torch.zeros(rows // 4, 4, device=DEV)
    out, parents, tokens = beam_select(z, s, 8)
    compare((out[-2:], parents[-2:], tokens[-2:]), tail, torch.zeros(2, 4), 8)
    assert (tokens[:-2, 0] == 0).all() and (parents[:-2, 0] == 0).all()
    assert tokens[0].tolist() == list(range(8)) and parents[0].tolist() == [0] * 8


@gpu
def test_selection_repeats_its_bits_on_any_stream_and_in_a_graph():
    z, s = rand((12, 20001), 19, "bf16"), rand((3, 4), 12)
    zd, sd = z.to(DEV), s.to(DEV)
    note("select streams and graphs")
    first = beam_select(zd, sd, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = beam_select(zd, sd, 8)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = beam_select(zd, sd, 8)
    for seed in (20, 21, 22):
        z = rand((12, 20001), seed, "bf16")
        zd.copy_(z)
        g.replay()
        torch.cuda.synchronize()
        compare(got, z, s, 8)
        for a, b in zip(got, beam_select(zd, sd, 8)):
            assert torch.equal(a, b)


@gpu
def test_two_selections_at_once():
    note("select two graphs")
    graphs = []
    for k, (requests, beams, vocab, keep) in enumerate([(9, 4, 30011, 8), (2, 7, 5003, 14)]):
        z = rand((requests * beams, vocab), 20 + k, "bf16").to(DEV)
        s = rand((requests, beams), 30 + k, sigma=1.0).to(DEV)
        eager = beam_select(z, s, keep)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = beam_select(z, s, keep)
        graphs.append((graph, eager, got, z, s))  # (a graph does not keep its inputs)
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for _, _, got, _, _ in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for side, (graph, *_) in zip(sides, graphs):
            with torch.cuda.stream(side):
                for _ in range(8):
                    graph.replay()
        torch.cuda.synchronize()
        for _, eager, got, _, _ in graphs:
            for p, q in zip(got, eager):
                assert torch.equal(p, q)


@gpu
def test_no_requests():
    got = beam_select(torch.zeros(0, 7, device=DEV), torch.zeros(0, 3, device=DEV), 4)
    assert [tuple(t.shape) for t in got] == [(0, 4)] * 3


# -- reordering on the GPU ----------------------------------------------------


def some_parents(requests, beams, seed, holes=True, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, beams, (requests, beams), generator=g)
    if holes:
        p[torch.rand(p.shape, generator=g) < 0.15] = -1
        p[torch.rand(p.shape, generator=g) < 0.05] = beams
    return p.to(dtype)


def some_state(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(shape, generator=g).to(dtype)
    return torch.randint(-100 if dtype != torch.uint8 else 0, 100, shape, generator=g).to(dtype)


def as_bytes(t):
    return t.contiguous().view(torch.uint8).numpy() if t.dtype == torch.bfloat16 else t.numpy()


def check_reorder(states, parents, lengths=None, time_dim=None):
    wants = []
    for t in states:
        idx = ob.beam_reorder(np.broadcast_to(np.arange(t.shape[0]).reshape(-1, *[1] * (t.dim() - 1)), t.shape),
                              parents.numpy(), None if lengths is None else lengths.numpy(),
                              None if time_dim is None else time_dim % t.dim())
        wants.append(t.gather(0, torch.from_numpy(idx)))
    device = [t.to(DEV) for t in states]
    beam_reorder(device if len(device) != 1 else device[0], parents.to(DEV),
                 None if lengths is None else lengths.to(DEV), time_dim)
    for t, want in zip(device, wants):
        assert torch.equal(t.cpu(), want)


@gpu
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float32, torch.int64])
@pytest.mark.parametrize("requests,beams,shape", [
    (1, 1, (5,)), (1, 2, (3, 5)), (3, 4, (2, 7, 33)), (2, 5, (1, 1, 1)), (4, 8, (3, 100, 16)), (2, 13, (2, 9, 5)),
    (3, 16, (1, 300, 7)), (2, 17, (2, 11, 3)), (1, 64, (3, 41, 9)), (5, 3, (0, 4, 4)), (1, 4, (1, 5000, 8))])
def test_reordering(dtype, requests, beams, shape):
    note(f"reorder {dtype} {requests} {beams} {shape}")
    t = some_state((requests * beams, *shape), beams, dtype)
    p = some_parents(requests, beams, beams + 1)
    check_reorder([t], p)
    dim = len(shape) - 1 if len(shape) > 1 else 1
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(-2, shape[dim - 1] + 3, (requests,), generator=g)
    check_reorder([t], p, lengths, dim)
    check_reorder([t], p.int(), lengths.int(), dim - 1 - len(shape))


@gpu
@pytest.mark.parametrize("beams", [2, 4, 7, 16, 40])
def test_cycles_and_copies(beams):
    t = some_state((2 * beams, 3, 50), beams)
    ring = torch.arange(beams).roll(1)
    for p in (ring, ring.flip(0), torch.arange(beams), torch.full((beams,), beams - 1), torch.arange(beams) // 2):
        note(f"reorder cycle {beams} {p.tolist()[:4]}")
        check_reorder([t], torch.stack([p, ring]))


@gpu
def test_many_states_in_one_call():
    # 70 of one geometry (two launches), then others in between
    p, lengths = some_parents(3, 4, 1), torch.tensor([0, 7, 31])
    states = [some_state((12, 2, 31, 5), k) for k in range(70)] + [some_state((12, 1, 40, 2), 71, torch.int64)]
    states += [some_state((12, 2, 31, 5), 72), some_state((12, 3, 33, 1), 73, torch.uint8)]
    note("reorder 73 states")
    check_reorder(states, p, lengths, 2)
    check_reorder([], p)


@gpu
def test_views_of_one_cache():
    note("reorder views")
    p, lengths = some_parents(2, 3, 2), torch.tensor([4, 9])
    cache = some_state((6, 2, 4, 9, 8), 4)  # rows, keys and values, heads, positions, channels
    want = torch.from_numpy(ob.beam_reorder(cache.numpy(), p.numpy(), lengths.numpy(), 3))
    d = cache.to(DEV)
    beam_reorder([d[:, 0], d[:, 1]], p.to(DEV), lengths.to(DEV), time_dim=2)
    assert torch.equal(d.cpu(), want)
    outside = some_state((4, 6, 9, 8), 5)  # heads outside of the rows
    want = torch.from_numpy(ob.beam_reorder(outside.transpose(0, 1).numpy(), p.numpy(), lengths.numpy(), 2))
    d = outside.to(DEV)
    beam_reorder(d.transpose(0, 1), p.to(DEV), lengths.to(DEV), time_dim=2)
    assert torch.equal(d.transpose(0, 1).cpu(), want)
    d = cache.to(DEV)
    with pytest.raises(HgError):
        beam_reorder([d[:, 0], d[:, :1]], p.to(DEV))
    with pytest.raises(HgError):
        beam_reorder([d, d], p.to(DEV))
    with pytest.raises(HgError):
        beam_reorder(d[:1].expand(6, 2, 4, 9, 8), p.to(DEV))
    assert torch.equal(d.cpu(), cache)


@gpu
@pytest.mark.parametrize("offset", [1, 2, 3, 4, 8, 12])
@pytest.mark.parametrize("beams", [4, 20])
def test_states_that_start_anywhere(offset, beams):
    note(f"reorder offset {offset} {beams}")
    t = some_state((2 * beams, 3, 77), offset, torch.uint8)
    room = torch.zeros(t.numel() + 64, dtype=torch.uint8, device=DEV)
    part = room[offset:offset + t.numel()].view(t.shape)
    part.copy_(t)
    p, lengths = some_parents(2, beams, offset), torch.tensor([77, 50])
    want = torch.from_numpy(ob.beam_reorder(t.numpy(), p.numpy(), lengths.numpy(), 2))
    beam_reorder(part, p.to(DEV), lengths.to(DEV), time_dim=2)
    assert torch.equal(part.cpu(), want)
    assert not room[:offset].any() and not room[offset + t.numel():].any()


@gpu
def test_reordering_past_32_bit_offsets():
    note("reorder 5 GB")
    t = torch.zeros(4, 1250, 1000003, dtype=torch.uint8, device=DEV)
    ends = torch.randint(1, 255, (4, 2), dtype=torch.uint8)
    t[:, 0, 0], t[:, -1, -1] = ends[:, 0].to(DEV), ends[:, 1].to(DEV)
    beam_reorder(t, torch.tensor([[3, 0, 0, 2]], device=DEV))
    order = [3, 0, 0, 2]
    assert torch.equal(t[:, 0, 0].cpu(), ends[order, 0]) and torch.equal(t[:, -1, -1].cpu(), ends[order, 1])


@gpu
def test_reordering_in_a_graph_and_on_a_side_stream():
    note("reorder graph")
    t, p = some_state((8, 3, 40, 6), 7), some_parents(2, 4, 8, holes=False)
    lengths = torch.tensor([40, 13])
    d, pd, ld = t.to(DEV), p.to(DEV), lengths.to(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam_reorder(d, pd, ld, time_dim=2)
    want = t.numpy()
    for seed in (9, 10, 11):
        p = some_parents(2, 4, seed)
        pd.copy_(p)
        g.replay()
        torch.cuda.synchronize()
        want = ob.beam_reorder(want, p.numpy(), lengths.numpy(), 2)
        assert (d.cpu().numpy() == want).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        beam_reorder(d, pd, ld, time_dim=2)
    side.synchronize()
    assert (d.cpu().numpy() == ob.beam_reorder(want, p.numpy(), lengths.numpy(), 2)).all()
