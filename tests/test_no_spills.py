"""The gated form of the skinny kernel stays inside its registers. A spilled vector register is
stored for the active lanes only, and the compiler has placed such a store ahead of the
restoring of the lanes' mask; so none may be spilled. Read from the compiled code's own
record at 6 and 8 bits, whose items are the largest."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from weight_only_quantized_qgemv_amd import _build


@pytest.mark.parametrize("bits", [6, 8])
def test_gated_kernels_spill_nothing(bits, tmp_path):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    asm = str(tmp_path / "gate_up.s")
    p = subprocess.run([_build.HIPCC, *_build.CFLAGS, f"-DQP_BITS={bits}", "--offload-device-only", "-S",
                        os.path.join(_build.CSRC, "gate_up.hip"), "-o", asm],
                       capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stderr
    with open(asm) as f:
        text = f.read()
    record = re.findall(r"\.name:\s+(_Z\w*kernel\w*).*?\.vgpr_spill_count:\s+(\d+)", text, re.S)
    assert sum("qgemv_skinny_kernel" in name for name, _ in record) == 6   # two types, three group sizes
    spilled = {name: int(n) for name, n in record if int(n)}
    assert not spilled, spilled
