"""qcross_entropy with small fp16 activations and weights so large that the logits are of the
usual size: the groups' sums of x, which meet the biases, keep their digits whatever their
size is. The bounds are those of test_gpu_loss.py: 2^-17 of a logit's magnitudes."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev, log
from test_gpu_loss import backward64, case, forward64

pytestmark = pytest.mark.gpu


def check(x, w, t, dloss, bits, gs, dt, what, backward=True):
    log(f"loss of small activations: {what}")
    wd, td = oh.cuda(w), t.to(dev())
    loss, lse = qp.qcross_entropy(x.to(dev()), td, *wd, bits, gs)
    torch.cuda.synchronize()
    (r_loss, b_loss), (r_lse, b_lse), _ = forward64(x, w, t, bits, gs, dt)
    oh.check(lse, r_lse, b_lse, f"{what} lse")
    oh.check(loss, r_loss, b_loss, f"{what} loss")
    if not backward:
        return
    grads = qp.qcross_entropy_backward(x.to(dev()), td, lse, dloss.to(dev()), *wd, bits, gs)
    torch.cuda.synchronize()
    for got, (ref, bound), name in zip(grads, backward64(x, w, t, lse.cpu(), dloss, bits, gs, dt), ("dx", "ds", "db")):
        oh.check(got, ref, bound, f"{what} {name}")


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("m,k,v,bits,gs", [(40, 256, 500, 4, 32), (40, 256, 500, 8, 64), (70, 4096, 300, 4, 64),
                                           (130, 2112, 260, 3, 32), (300, 8320, 257, 6, 128), (9, 256, 500, 4, 32),
                                           (33, 20480, 70, 2, 32)])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -13])
def test_small_rows(size, m, k, v, bits, gs, dt):
    """Activations of 1e-3 and 1e-4, weights of 2^9 times the usual ones (a multiple of the codes'
    and biases' own rounding, so that they stay exact)."""
    x, (wq, s, b), t, dloss = case(m, k, v, bits, gs, dt, sigma=size)
    w = (wq, s * 2.0 ** 9, b * 2.0 ** 9)
    assert torch.isfinite(w[1]).all() and torch.isfinite(w[2]).all()
    check(x, w, t, dloss, bits, gs, dt, f"m={m} k={k} v={v} bits={bits} gs={gs} dt={dt} size={size}")


@pytest.mark.parametrize("m,k,v,gs", [(20, 320, 400, 32), (69, 384, 400, 64), (200, 128, 32003, 32),
                                      (200, 128, 32003, 128), (600, 128, 33001, 64), (600, 96, 33001, 32)])
def test_rows_of_every_size_together(m, k, v, gs):
    """Neighbouring rows' activations are powers of two apart, from 2^12 to 2^-10, one row of zeros:
    each row keeps its own digits, in the tiles of 32 to 256 rows."""
    bits = 4
    x, w, t, dloss = case(m, k, v, bits, gs, F16, sigma=1.0)
    x = (x.float() * (2.0 ** (12.0 - torch.arange(m) % 23))[:, None]).to(x.dtype)
    x[5] = 0
    assert torch.isfinite(x).all()
    check(x, w, t, dloss, bits, gs, F16, f"sizes together m={m} v={v} gs={gs}", backward=False)


def test_largest_sums():
    """Groups of 128 values of fp16's largest: their sums are 128 times its range."""
    m, k, v, bits, gs = 40, 512, 300, 4, 128
    x, (wq, s, b), t, dloss = case(m, k, v, bits, gs, F16)
    x[:] = 65504.0
    x[1::2] = -65504.0
    w = (wq, s * 2.0 ** -13, b * 2.0 ** -13)
    check(x, w, t, dloss, bits, gs, F16, "largest", backward=False)
