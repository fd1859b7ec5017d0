"""The record of which kernels may use their dynamic LDS on which device (allow_lds in
csrc/launch.hpp), on the CPU under ThreadSanitizer: four devices, sixteen threads."""
from __future__ import annotations

import os
import subprocess

import pytest

SAN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")
HIPCC = "/opt/rocm/bin/hipcc"


def test_every_device_is_asked(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "lds_driver")
    p = subprocess.run([HIPCC, "--offload-arch=gfx950", "-x", "hip", "-std=c++17", "-O1", "-g",
                        "-Xarch_host", "-fsanitize=thread", os.path.join(SAN, "lds_driver.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "asked once per device" in p.stdout, p.stdout + p.stderr
