"""Spans from offsets that only the device sees (csrc/span.hpp), on the CPU: every
combination of extreme offsets and list lengths, with overflow trapped."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

SAN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")


def test_spans_stay_inside_their_list(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "span_driver")
    p = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        os.path.join(SAN, "span_driver.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and "all spans inside" in p.stdout, p.stdout + p.stderr
