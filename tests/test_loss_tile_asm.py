"""What the loss's tile kernels rely on in their compiled code. A step ends with a counted
wait: all loads have landed but those for the steps after the next two (with four stages of
codes and scales those of the step itself; the tiles of 32 and 64 rows have up to eight stages), so
each step has to issue exactly the loads that its source counts, the activations' first. And none of the kernels spills a vector
register: a spill is stored for the active lanes only, and the compiler has placed such a
store where the lanes' mask was partial."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from weight_only_quantized_qgemv_amd import _build


@pytest.fixture(scope="module", params=[3, 4, 6, 8])
def asm(request, tmp_path_factory):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "loss_tile.s")
    p = subprocess.run([_build.HIPCC, *_build.CFLAGS, f"-DQP_BITS={request.param}", "--offload-device-only", "-S",
                        os.path.join(_build.CSRC, "loss_tile.hip"), "-o", out],
                       capture_output=True, text=True, timeout=900)
    assert p.returncode == 0, p.stderr
    with open(out) as f:
        return request.param, f.read()


def test_tile_kernels_spill_nothing(asm):
    _, text = asm
    record = re.findall(r"\.name:\s+(_Z\w*loss_tile_kernel\w*).*?\.vgpr_spill_count:\s+(\d+)", text, re.S)
    assert len(record) == 24    # three types, four tiles, groups of 32 and larger ones
    assert not {name: n for name, n in record if int(n)}


def test_steps_issue_the_loads_that_their_ends_count(asm):
    bits, text = asm
    kernels = re.findall(r"^_ZN2qp8losstile16loss_tile_kernelILi\d+ELi(\d)ELi(\d)ELi(\d)ELb(\d)E\S+:(.*?)^\s+s_endpgm$",
                         text, re.S | re.M)
    kernels = [(int(dt), int(fm), int(wmw), int(g32), body) for dt, fm, wmw, g32, body in kernels]
    assert len(kernels) == 24
    for dt, fm, wmw, g32, body in kernels:
        waves = 4 * wmw
        a_loads = 32 * fm * wmw * 128 // 1024 // waves
        chunk = 12 if bits == 3 else 16
        slots = 256 * 8 * bits // chunk             # a step's codes: 256 rows of 64
        codes = -(-slots // (64 * waves))
        fp32 = dt == 0
        scales = -(-(4 if fp32 else 2) * (2 if g32 else 1) // waves)
        # (A product that ends a step may stand behind its barrier.)
        parts = [b for b in body.split("s_barrier") if "v_mfma_f32_32x32x16" in b]
        assert sum(b.count("v_mfma_f32_32x32x16") for b in parts) == 8 * fm * (1 if fp32 else 2)
        steps = [b for b in parts if re.search(r"\bbuffer_load_\w+[^\n]* lds\b", b)]
        assert len(steps) == (1 if fp32 else 2), (bits, dt, fm, wmw, g32)    # the codes'; the biases' of 16-bit types
        for step in steps:
            staged = re.findall(r"\bbuffer_load_\w+[^\n]* lds\b", step)
            assert len(staged) == a_loads + codes + scales, (bits, dt, fm, wmw, g32, staged)
            last = [k for k in re.findall(r"\bbuffer_load_[^\n]*", step)][-(codes + scales):]
            assert all(k.rstrip().endswith("lds") for k in last)
            assert sum("dwordx" in k for k in last) == codes
            waits = [int(n) for n in re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", step)]
            if fm <= 2:
                stage = 4096 * fm + 4096 * codes + 1024 * scales
                ahead = (min(max(80 * 1024 // stage, 3), 8) - 3) * len(staged)
            else:
                ahead = codes + scales if bits < 6 else 0
            assert waits[-1] == ahead, (bits, dt, fm, wmw, g32, waits)
