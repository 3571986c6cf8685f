"""The compiled kernels of the cross entropy: their loads into LDS are written
as instructions, so the compiler does not put the wait states that such a load
needs behind a vector instruction that writes one of its scalar registers. None
may stand that close (CPU: compiles to assembly)."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from tp_vocab_logits_amd import build

NEEDED = 5  # wait states between a vector write of a scalar register and a vector memory read of it


def written(line: str) -> set[int]:
    """Scalar registers that a vector instruction writes."""
    m = re.match(r"v_\w+ (?:v\S+, )?s(?:\[(\d+):(\d+)\]|(\d+)\b)", line)
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def loads_too_close(lines: list[str]) -> tuple[int, list[list[str]]]:
    """Number of loads into LDS, and the runs of lines that end in one whose
    resource was written fewer than NEEDED wait states before."""
    count, bad = 0, []
    for k, line in enumerate(lines):
        m = re.match(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\], .*\blds$", line)
        if not m:
            continue
        count += 1
        need, states = set(range(int(m[1]), int(m[2]) + 1)), 0
        for j in range(k - 1, -1, -1):
            if states >= NEEDED:
                break
            if written(lines[j]) & need:
                bad.append(lines[j:k + 1])
                break
            nop = re.match(r"s_nop (\d+)", lines[j])
            states += int(nop[1]) + 1 if nop else 0 if lines[j].endswith(":") else 1
    return count, bad


def test_the_check_sees_a_close_write():
    load = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"
    assert loads_too_close(["v_readfirstlane_b32 s9, v3", "s_mov_b32 m0, s2", "s_nop 0", load])[1]
    assert loads_too_close(["v_cmp_gt_i32_e64 s[10:11], v1, v2", load])[1]
    assert not loads_too_close(["v_readfirstlane_b32 s9, v3", "s_nop 4", load])[1]
    assert not loads_too_close(["v_readfirstlane_b32 s12, v3", load])[1]
    assert loads_too_close([load])[0] == 1


def test_resources_are_written_early_enough(tmp_path):
    out = str(tmp_path / "hg_xent.s")
    cmd = build.compile_command("hg_xent.hip", out)
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    cmd[cmd.index("-c")] = "-S"
    res = subprocess.run([*cmd, "--cuda-device-only"], capture_output=True, text=True)
    assert res.returncode == 0 and os.path.exists(out), res.stderr[-2000:]
    lines = [ln.split(";")[0].strip() for ln in open(out)]
    lines = [ln for ln in lines if ln and not ln.startswith((".", "#")) or ln.endswith(":")]
    count, bad = loads_too_close(lines)
    assert count > 100
    assert not bad, bad[:3]
