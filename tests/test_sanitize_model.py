"""The host side of the operators around the products (api_model.cpp, on
api.cpp's shared checks) built with AddressSanitizer and
UndefinedBehaviorSanitizer and run on the CPU by
tests/sanitize/model_driver.cpp, whose launchers only count their calls."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "weight_only_quantized_qgemv_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


def test_model_abi_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "model_driver")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    p = subprocess.run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", *san,
                        os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "api_model.cpp"),
                        os.path.join(SAN, "abi_stubs.cpp"), os.path.join(SAN, "model_driver.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    # Leak checking is off: the HIP runtime's own start-up allocations would
    # be reported.
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert p.returncode == 0 and "all calls clean" in p.stdout, p.stdout + p.stderr
