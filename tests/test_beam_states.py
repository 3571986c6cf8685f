"""Which states hg_beam_reorder takes together: those that share no byte, also between each other's rows, and in how much
time it finds out (CPU: every call here ends in a refusal, the last one of a state larger than a launch covers, so
that nothing is launched)."""

from __future__ import annotations

import itertools
import random
import time

import pytest

from tp_vocab_logits_amd import _lib

REQUESTS = 4  # of one beam
HUGE = _lib.BeamState(1 << 60, 1 << 43, 0, 1 << 32, 1, 1 << 10)
TAKEN, OVERLAP = "more runs of rows than a launch covers", "overlap"


def answer(states, requests=REQUESTS):
    a = (_lib.BeamState * (len(states) + 1))(*states, HUGE)
    code = _lib.lib().hg_beam_reorder(requests, 1, len(a), a, 1 << 59, 8, None, 8, None)
    assert code == _lib.HG_EINVAL
    return _lib.lib().hg_last_error_detail().decode()


def state(at, row, outer_stride, run, outer):
    return _lib.BeamState((1 << 40) + at, row, outer_stride, run, outer, 1)


def bytes_of(s, rows=REQUESTS):
    return {s.ptr + r * s.row_stride + o * s.outer_stride + b
            for r, o, b in itertools.product(range(rows), range(s.outer), range(s.step_bytes))}


def test_the_last_refusal_is_the_launchs():
    assert TAKEN in answer([])
    assert TAKEN in answer([state(0, 10, 0, 10, 1)])
    assert OVERLAP in answer([state(0, 9, 0, 10, 1)])
    assert OVERLAP in answer([state(0, 10, 0, 10, 1)] * 2)


def some_state(rng, rows_inside):
    run, outer = rng.randint(1, 4), rng.choice([1, 2, 3])
    small = run + rng.randint(0, 9)
    large = small * (outer if not rows_inside else REQUESTS) + rng.randint(0, 12)
    return (small, large, run, outer) if rows_inside else (large, small, run, outer)


@pytest.mark.parametrize("seed", range(40))
def test_two_states_against_their_bytes(seed):
    """Those that share a byte are refused, those of one geometry that share none are taken."""
    rng = random.Random(seed)
    taken = 0
    for _ in range(60):
        row, step, run, outer = some_state(rng, rng.random() < 0.3)
        a = state(rng.randint(0, 60), row, step, run, outer)
        alike = rng.random() < 0.6
        b = state(rng.randint(0, 60), row, step, run if alike else rng.randint(1, 4), outer if alike else rng.choice([1, 2]))
        got = answer([a, b])
        assert answer([b, a]) == got
        if bytes_of(a) & bytes_of(b) or len(bytes_of(b)) < REQUESTS * b.outer * b.step_bytes:
            assert OVERLAP in got, (a.ptr, b.ptr, row, step, run, outer, b.step_bytes, b.outer)
        elif alike:
            assert TAKEN in got, (a.ptr, b.ptr, row, step, run, outer)
            taken += 1
    assert taken > 5


@pytest.mark.parametrize("seed", range(20))
def test_many_states_against_their_bytes(seed):
    """Views of one cache, in any order, some of them of another width; then one byte of one of them moved."""
    rng = random.Random(100 + seed)
    inside, views, heads = rng.random() < 0.5, rng.randint(2, 7), rng.randint(1, 3)
    widths = [rng.randint(1, 5) for _ in range(views)] if rng.random() < 0.5 else [3] * views
    starts = [sum(widths[:k]) for k in range(views)]
    if inside:  # [row, head, view, channel]
        row, step = heads * sum(widths), sum(widths)
        states = [state(at, row, step, w, heads) for at, w in zip(starts, widths)]
    else:  # [row, view, head, channel]
        row = heads * sum(widths)
        states = [state(heads * at, row, w, w, heads) for at, w in zip(starts, widths)]
    rng.shuffle(states)
    assert TAKEN in answer(states)
    k = rng.randrange(views)
    s = states[k]
    for by in (1, -1):
        moved = [*states[:k], _lib.BeamState(s.ptr + by, s.row_stride, s.outer_stride, s.step_bytes, s.outer, 1), *states[k + 1:]]
        others = set().union(*(bytes_of(t) for t in states[:k] + states[k + 1:]))
        assert (OVERLAP in answer(moved)) == bool(bytes_of(moved[k]) & others)


def test_keys_and_values_of_different_width_in_one_row():
    row = 4 * 128 + 4 * 64
    keys, values = state(0, row, 128, 128, 4), state(4 * 128, row, 64, 64, 4)
    assert TAKEN in answer([keys, values])
    assert OVERLAP in answer([keys, state(4 * 128 - 1, row, 64, 64, 4)])
    assert OVERLAP in answer([keys, state(4 * 128 + 1, row, 64, 64, 4)])


@pytest.mark.parametrize("inside", [False, True])
def test_many_views_take_little_time(inside):
    """4096 views of one cache, 128 heads: pairs of them head by head were 10^9 divisions."""
    views, heads, run = 4096, 128, 256
    row = views * heads * run
    states = [state(k * run, row, views * run, run, heads) if inside else state(k * heads * run, row, run, run, heads)
              for k in range(views)]
    begin = time.process_time()
    assert TAKEN in answer(states)
    assert OVERLAP in answer([*states[:-1], states[7]])
    assert time.process_time() - begin < 2.0
    # a state of the most runs beside another one in its gaps
    begin = time.process_time()
    many = [state(k * 16, 1 << 28, 64, 16, 1 << 20) for k in range(4)]
    assert TAKEN in answer(many)
    assert OVERLAP in answer([*many, state(63, 1 << 28, 64, 16, 1 << 20)])
    assert time.process_time() - begin < 0.5
