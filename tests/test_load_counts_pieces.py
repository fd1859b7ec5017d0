"""The gradient products' kernels as the loss calls them (sums kept over pieces of the
contraction, results times a factor) are compiled apart from those that qmatmul_backward and
qffn_backward call, whose code has none of it; their steps issue the loads that their ends
count, as the others' do (test_load_counts.py)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from weight_only_quantized_qgemv_amd import _build
from test_load_counts import STEP


def assembly(tmp_path, source, *defines):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    asm = str(tmp_path / "out.s")
    p = subprocess.run([_build.HIPCC, *_build.CFLAGS, *defines, "--offload-device-only", "-S",
                        os.path.join(_build.CSRC, source), "-o", asm], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stderr
    with open(asm) as f:
        return f.read()


@pytest.mark.parametrize("bits", [3, 6])
def test_the_steps_of_the_pieces_kernels(bits, tmp_path):
    text = assembly(tmp_path, "xgrad.hip", f"-DQP_BITS={bits}", "-DQP_PIECES=1")
    kernels = re.findall(r"^_ZN2qp8gradtile17xgrad_tile_kernel\S+Lb1E\S+:.*?s_endpgm", text, re.S | re.M)
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


@pytest.mark.parametrize("source,define", [("xgrad.hip", "-DQP_PIECES=1"), ("wgrad.hip", "-DQP_SCALED=1")])
def test_the_two_builds_share_no_kernel(source, define, tmp_path):
    names = [set(re.findall(r"^(_ZN2qp\w*grad\w*kernel\w*):", assembly(tmp_path, source, "-DQP_BITS=4", *d), re.M))
             for d in ((), (define,))]
    assert names[0] and names[1] and not names[0] & names[1]
    assert all("Lb0E" in n for n in names[0]) and all("Lb1E" in n for n in names[1])
