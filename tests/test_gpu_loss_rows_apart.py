"""qcross_entropy and its backward pass: what is in one row of x reaches no other row's loss, lse
or dx, in any type."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev
from test_gpu_loss import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf", "large"])
@pytest.mark.parametrize("m,k,v,gs", [(2, 256, 700, 32), (4, 256, 700, 32), (16, 256, 700, 64), (70, 256, 700, 32),
                                      (300, 256, 700, 64), (20, 32, 700, 32), (200, 64, 33000, 32), (600, 64, 33000, 64)])
def test_the_other_rows_keep_their_bits(m, k, v, gs, bad, dt):
    x, w, t, dloss = case(m, k, v, 4, gs, dt)
    t[:] = 5
    wd, td, gd = oh.cuda(w), t.to(dev()), dloss.to(dev())
    at = m // 2
    other = x.clone()
    other[at, k - 1] = 60000.0 if bad == "large" else float(bad)
    runs = []
    for xx in (x, other):
        loss, lse = qp.qcross_entropy(xx.to(dev()), td, *wd, 4, gs)
        back = qp.qcross_entropy_backward(xx.to(dev()), td, lse, gd, *wd, 4, gs, weight_grads=False)[0]
        runs.append((loss, lse, back))
    torch.cuda.synchronize()
    keep = [i for i in range(m) if i != at]
    for a, b in zip(*runs):
        assert oh.same_bits(a[keep], b[keep])
        if bad != "large":
            assert b[at].isnan().all()
