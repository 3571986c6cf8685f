"""The compiled scan of the beam selection: of a beam that is finished or not there no logit is read, so every load of
them (the only ones past the caches) stands behind the load of the flag that says so (CPU: compiles to assembly)."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from tp_vocab_logits_amd import build


def kernels(text: str) -> dict[str, list[str]]:
    out, name = {}, None
    for line in text.splitlines():
        start = re.match(r"(_ZN\w*k_beam_scan\w*):", line)
        if start:
            name = start[1]
            out[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            out[name].append(line.split(";")[0].strip())
    return out


def reads_first(lines: list[str]) -> bool:
    flag = [k for k, ln in enumerate(lines) if ln.startswith("global_load_ubyte ")]
    logits = [k for k, ln in enumerate(lines) if re.match(r"global_load_dword\w* .*\bnt$", ln)]
    branch = [k for k, ln in enumerate(lines) if ln.startswith("s_cbranch")]
    return bool(logits) and bool(flag) and any(flag[0] < k < logits[0] for k in branch)


def test_the_check_sees_an_early_read():
    flag, leave, logits = "global_load_ubyte v1, v1, s[4:5]", "s_cbranch_vccnz .L1", "global_load_dwordx4 v[2:5], v[2:3], off nt"
    assert reads_first([flag, leave, logits, logits])
    assert not reads_first([logits, flag, leave, logits])
    assert not reads_first([flag, logits, leave])
    assert not reads_first([flag, leave])


def test_absent_beams_are_left_before_their_logits(tmp_path):
    out = str(tmp_path / "hg_beam.s")
    cmd = build.compile_command("hg_beam.hip", out)
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    cmd[cmd.index("-c")] = "-S"
    res = subprocess.run([*cmd, "--cuda-device-only"], capture_output=True, text=True)
    assert res.returncode == 0 and os.path.exists(out), res.stderr[-2000:]
    found = kernels(open(out).read())
    assert len(found) == 27  # three types, three sizes of a part, three of the table
    assert [name for name, lines in found.items() if not reads_first(lines)] == []
