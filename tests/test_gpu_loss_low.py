"""qcross_entropy and its backward pass where all logits of a row are far below or above 0, at
vocabularies with fewer logits than a block has threads and more: a share of a row without any
logit must not take part in its maximum. The bounds are those of test_gpu_loss.py; S is about
the level itself there, since the biases carry it."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev, log
from test_gpu_loss import backward64, case, forward64

pytestmark = pytest.mark.gpu


def at_level(m, k, v, dt, level):
    """A case whose logits are about `level`: x about 1, the biases level / k."""
    x, (wq, s, b), t, dloss = case(m, k, v, 4, 32, dt)
    x = (1 + 0.125 * x.float()).to(x.dtype)
    return x, (wq, s, (b.float() + level / k).to(b.dtype)), t, dloss


def check(m, k, v, dt, level):
    log(f"loss of low logits: m={m} k={k} v={v} dt={dt} level={level}")
    x, w, t, dloss = at_level(m, k, v, dt, level)
    wd, td = oh.cuda(w), t.to(dev())
    loss, lse = qp.qcross_entropy(x.to(dev()), td, *wd, 4, 32)
    torch.cuda.synchronize()
    (r_loss, b_loss), (r_lse, b_lse), (z, *_) = forward64(x, w, t, 4, 32, dt)
    assert (z < 0).all() if level < 0 else (z > 0).all()
    oh.check(lse, r_lse, b_lse, f"level {level} lse")
    oh.check(loss, r_loss, b_loss, f"level {level} loss")
    grads = qp.qcross_entropy_backward(x.to(dev()), td, lse, dloss.to(dev()), *wd, 4, 32)
    torch.cuda.synchronize()
    for got, (ref, bound), name in zip(grads, backward64(x, w, t, lse.cpu(), dloss, 4, 32, dt), ("dx", "ds", "db")):
        oh.check(got, ref, bound, f"level {level} {name}")


# 16-bit rows of the decode kernels; fp32 rows that are too short for the tiles.
@pytest.mark.parametrize("k,dt", [(64, F16), (64, BF16), (32, F32)])
@pytest.mark.parametrize("v", [1, 5, 40, 256, 700, 1000, 2048, 4092, 4093, 5000])
@pytest.mark.parametrize("m", [1, 2, 16])
def test_few_rows(m, v, k, dt):
    for level in (-100.0, -150.0, -500.0, 150.0):
        check(m, k, v, dt, level)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,k,v", [(40, 64, 5), (40, 64, 300), (40, 32, 700), (40, 32, 4097), (3, 64, 66000), (300, 128, 257)])
def test_other_paths(m, k, v, dt):
    """The tiles, and the parts of rows that go without them."""
    for level in (-150.0, -500.0, 150.0):
        check(m, k, v, dt, level)
