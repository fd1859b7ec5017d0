"""Gradients of qblock_norm for rows far smaller and far larger than 1, down to eps = 0: no
power of 1 / rms beyond what the result itself is of is formed. The bounds are those of
test_gpu_norm.py."""
from __future__ import annotations

import pytest

import test_gpu_norm
from qhelpers import BF16, F32
from test_gpu_norm import Case, run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,sdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", [100, 1000, 5000, 8200])
@pytest.mark.parametrize("size", [1e-15, 1e-13, 1e13, 1e15])
def test_rows_far_from_1(monkeypatch, size, d, dt, sdt):
    """The squares, 1e-30 and 1e33 at most, and the gradients, 1e15 times their upstream ones, are
    inside fp32's range; a cube of 1 / rms is not."""
    monkeypatch.setattr(test_gpu_norm, "EPS", 0.0)
    c = Case(7, d, dt, sdt, False, 0, True, y=False)
    c.x = (c.x.float() * size).to(c.x.dtype)
    run_and_check(c, f"stream of {size}")
    c = Case(7, d, dt, sdt, True, 1, False)
    c.y = (c.y.float() * size).to(c.y.dtype)
    run_and_check(c, f"block of {size}")
