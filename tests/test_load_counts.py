"""The input gradient's tile kernel ends a step with a counted wait: all loads but those the
step itself issued have landed. The count is a constant of the source, so each step of the
compiled code has to issue exactly that many loads; one merged by the compiler would let
the wait pass before the next step's tile is there. Counted in the assembly of the widths
whose octets take two words, where a merge is possible (a row's words are one load by the
source's own form at 6 bits and have separate offsets at 3)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from weight_only_quantized_qgemv_amd import _build

STEP = re.compile(r"^\.LBB\S+:", re.M)


@pytest.mark.parametrize("bits", [3, 6])
def test_a_step_issues_the_loads_that_its_end_counts(bits, tmp_path):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    asm = str(tmp_path / "xgrad.s")
    p = subprocess.run([_build.HIPCC, *_build.CFLAGS, f"-DQP_BITS={bits}", "--offload-device-only", "-S",
                        os.path.join(_build.CSRC, "xgrad.hip"), "-o", asm],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    with open(asm) as f:
        text = f.read()
    kernels = re.findall(r"^_ZN2qp8gradtile17xgrad_tile_kernel\S+:.*?s_endpgm", text, re.S | re.M)
    assert len(kernels) == 6    # two types, three tiles
    for body in kernels:
        steps = [b for b in STEP.split(body) if "v_mfma" in b and "s_barrier" in b]
        assert len(steps) == 2  # the two stages
        for step in steps:
            to_barrier = step[:step.index("s_barrier")]
            loads = len(re.findall(r"\bbuffer_load_\w+", to_barrier))
            waits = [int(n) for n in re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", to_barrier)]
            assert waits and waits[-1] == loads, (loads, waits)
            singles = len(re.findall(r"\bbuffer_load_dword\b", to_barrier))
            assert singles == (0 if bits == 6 else 8)
