"""Gradients of qcross_entropy where a row's probability is all in one or two tokens: dx is then
one or two rows of the weight, and nothing averages out. Its 16-bit roundings are three, each
of half a step at most: dz's, the weight's and dx's own. So in place of TAU, which takes the
weights' roundings as averaged, the bound has HALF_ULP |dz| |W| for them, and the second order
of the two together; the others are those of test_gpu_loss.py."""
from __future__ import annotations

import pytest
import torch

import test_gpu_loss
import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, HALF_ULP, dev, log
from test_gpu_loss import backward64, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,k,v,bits,gs", [(1, 256, 700, 4, 64), (16, 512, 900, 8, 32), (75, 256, 700, 3, 32),
                                           (524, 256, 677, 8, 64), (300, 1024, 2000, 4, 128), (40, 128, 30, 4, 32)])
def test_peaked_rows(monkeypatch, m, k, v, bits, gs, dt):
    log(f"peaked rows: m={m} k={k} v={v} bits={bits} gs={gs} dt={dt}")
    # dx's products are fp32 sums over v tokens: (v + 64) 2^-24 beside the weight's rounding.
    tau = (0.0 if dt == F32 else HALF_ULP[dt] * (1 + HALF_ULP[dt])) + oh.gamma(v)
    monkeypatch.setattr(test_gpu_loss, "TAU", {dt: tau})
    x, w, t, dloss = case(m, k, v, bits, gs, dt, sigma=30.0)
    dloss = dloss * 2.0 ** -6    # (fp16: the scales' sums of up to 255 x stay in range)
    xd, td, wd = x.to(dev()), t.to(dev()), oh.cuda(w)
    _, lse = qp.qcross_entropy(xd, td, *wd, bits, gs)
    out = qp.qcross_entropy_backward(xd, td, lse, dloss.to(dev()), *wd, bits, gs)
    torch.cuda.synchronize()
    for got, (ref, bound), name in zip(out, backward64(x, w, t, lse.cpu(), dloss, bits, gs, dt), ("dx", "ds", "db")):
        oh.check(got, ref, bound, f"peaked {name}")
