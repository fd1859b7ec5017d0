"""The gated block's launches stay inside the workspace that is asked for, whatever the sizes,
widths and alignments (tests/sanitize/ffn_room_driver.cpp), on the CPU."""
from __future__ import annotations

import os
import subprocess

import pytest

from weight_only_quantized_qgemv_amd import _build

SAN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")


def test_launches_stay_inside_the_workspace(tmp_path):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "ffn_room_driver")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    p = subprocess.run([_build.HIPCC, "--offload-arch=gfx950", "-x", "hip", "-std=c++17", "-O1", "-g", *san,
                        os.path.join(SAN, "ffn_room_driver.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert p.returncode == 0 and "all inside the workspace" in p.stdout, p.stdout[-2000:] + p.stderr[-4000:]
