"""Calls of more threads than one grid dimension takes (2^32), in sizes that fit the GPU."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import F16, dev, log

pytestmark = pytest.mark.gpu


def need(gib):
    if torch.cuda.get_device_properties(0).total_memory < gib * 2 ** 30 * 1.1:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_embedding_of_more_than_2_24_tokens():
    """2^24 tokens of 2048 columns, 64 GiB: compared slice by slice with calls of a few tokens."""
    need(80)
    t, v, k, bits, gs = 2 ** 24 + 5, 97, 2048, 2, 128
    log(f"lookup of {t} tokens of {k}")
    w = oh.cuda(oh.weight(v, k, bits, gs, F16, oh.rng(1)))
    ids = (torch.arange(t, dtype=torch.int64, device=dev()) * 31 % (v + 1)).to(torch.int32)   # id v: zeros
    rows = qp.qembedding(torch.arange(v + 1, dtype=torch.int32, device=dev()), *w, bits, gs, 2.0)
    out = qp.qembedding(ids, *w, bits, gs, 2.0)
    step = 2 ** 20
    for at in range(0, t, step):
        part = ids[at:at + step].long()
        assert torch.equal(out[at:at + step].view(torch.int16), rows.view(torch.int16)[part]), at
    del out


@pytest.mark.parametrize("same", [False, True])
def test_embedding_gradient_of_2_27_tokens(same):
    """2^27 + 2049 tokens: sums of ones, exact in fp32 below 2^24 each. With one id for most
    tokens a single run crosses most windows."""
    need(60)
    t, v, k, bits, gs = 2 ** 27 + 2049, 4001, 32, 8, 32
    log(f"embedding gradient of {t} tokens, one id: {same}")
    g = torch.Generator(device="cuda").manual_seed(5)
    wq = torch.zeros((v, k * bits // 32), dtype=torch.int32, device=dev())
    wq[:, 0] = 3                                  # column 0 has code 3, the others 0
    ids = torch.randint(-1, v + 1, (t,), generator=g, device=dev(), dtype=torch.int32)
    if same:
        ids[torch.rand(t, generator=g, device=dev()) < 0.9] = 77
    live = (ids >= 0) & (ids < v)
    count = torch.bincount(ids[live].long(), minlength=v).double()
    # Every token adds 2^-10 at column 0: sums of up to 2^27 tokens, fp32 partial sums in order.
    dout = torch.zeros((t, k), dtype=torch.bfloat16, device=dev())
    dout[:, 0] = 2.0 ** -10
    ds, db = qp.qembedding_backward(ids, dout, wq, bits, gs)
    for got, want in ((ds, 3 * count * 2.0 ** -10), (db, count * 2.0 ** -10)):
        bound = want * 2.0 ** -8 + want * oh.gamma(64)   # half an ulp of bf16, and partial sums of windows
        assert ((got[:, 0].double() - want).abs() <= bound).all()


def test_logits_of_more_than_2_23_rows():
    rows, v = 2 ** 23 + 3, 32
    log(f"logits of {rows} rows of {v}")
    z = torch.arange(rows * v, device=dev(), dtype=torch.int32).remainder(251).to(torch.bfloat16).view(rows, v)
    mask = torch.tensor([[0x7FFFFFFE]], dtype=torch.int32, device=dev())
    out = qp.qlogits_adjust(z, mask=mask)
    assert torch.equal(out[:, 1:31], z[:, 1:31])
    assert (out[:, 0] == float("-inf")).all() and (out[:, 31] == float("-inf")).all()
