"""Host-side checks of the operators that train and score a model (no GPU needed): every
argument error is reported with its status and a message before any HIP call, calls
with nothing to do succeed, and workspace sizes are 0 for what is refused."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
from test_abi_model import (A, ALIGN, BF16, BIG, F16, F32, INVALID, LAYOUT, MISMATCH, ODD, OK, P, SHAPE, UNSUPPORTED,
                            WORKSPACE, refused)

HALF = P(0x10002)   # off a 4-byte address
NAN, INF = float("nan"), float("inf")


def loss(x=A, dt=BF16, m=2, k=128, t=A, w=(A, A, A), sdt=None, v=40, bits=4, gs=64, out=A, lse=A, ws=A, nws=1 << 40):
    return qp.lib().qcross_entropy(x, dt, m, k, t, *w, dt if sdt is None else sdt, v, bits, gs, out, lse, ws, nws, None)


LOSS = LAYOUT + [
    (dict(k=96), SHAPE), (dict(m=-1), INVALID), (dict(k=-64), INVALID), (dict(v=-1), INVALID), (dict(dt=3), INVALID),
    (dict(sdt=F16), MISMATCH), (dict(m=BIG), INVALID), (dict(m=(1 << 20) + 1), INVALID), (dict(k=BIG), INVALID),
    (dict(v=BIG), INVALID), (dict(x=None), INVALID), (dict(x=ODD), ALIGN), (dict(t=None), INVALID),
    (dict(t=HALF), ALIGN), (dict(lse=None), INVALID), (dict(lse=HALF), ALIGN), (dict(w=(None, A, A)), INVALID),
    (dict(w=(A, None, A)), INVALID), (dict(w=(A, A, ODD)), ALIGN), (dict(w=(HALF, A, A)), ALIGN),
    (dict(ws=None), INVALID), (dict(nws=16), WORKSPACE), (dict(ws=P(0x10008)), ALIGN),
]


@pytest.mark.parametrize("kw,status", LOSS + [
    (dict(out=None), INVALID), (dict(out=HALF), ALIGN),
    (dict(m=0, x=None, t=None, out=None, lse=None, ws=None), OK)])
def test_qcross_entropy(kw, status):
    refused(loss(**kw), status)


def loss_backward(x=A, dt=BF16, m=2, k=128, t=A, lse=A, dloss=A, w=(A, A, A), sdt=None, v=40, bits=4, gs=64, dx=A,
                  ds=A, db=A, ws=A, nws=1 << 40):
    return qp.lib().qcross_entropy_backward(x, dt, m, k, t, lse, dloss, *w, dt if sdt is None else sdt, v, bits, gs, dx,
                                            ds, db, ws, nws, None)


@pytest.mark.parametrize("kw,status", LOSS + [
    (dict(dloss=None), INVALID), (dict(dloss=HALF), ALIGN), (dict(dx=ODD), ALIGN), (dict(ds=ODD), ALIGN),
    (dict(ds=None), INVALID), (dict(db=None), INVALID),
    (dict(dx=None, ds=None, db=None, x=None, t=None, lse=None, ws=None), OK)])
def test_qcross_entropy_backward(kw, status):
    refused(loss_backward(**kw), status)


def norm(x=A, sdt=BF16, m=6, d=100, y=A, dt=BF16, w=A, post=A, gate=None, rows=0, scale=1.0, offset=0.0, eps=1e-6,
         s=A, out=A):
    return qp.lib().qblock_norm(x, sdt, m, d, y, dt, w, post, gate, rows, scale, offset, eps, s, out, None)


NORM = [
    (dict(m=-1), INVALID), (dict(d=-1), INVALID), (dict(dt=3), INVALID), (dict(sdt=-1), INVALID),
    (dict(sdt=F16), MISMATCH), (dict(dt=F32), MISMATCH), (dict(d=16385), UNSUPPORTED), (dict(m=BIG), INVALID),
    (dict(gate=A, rows=4), SHAPE), (dict(gate=A, rows=0), SHAPE), (dict(gate=A, rows=-1), SHAPE),
    (dict(gate=A, rows=12), SHAPE), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(offset=NAN), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(y=None, w=None, post=None), INVALID), (dict(y=None), INVALID),
    (dict(y=None, post=None, gate=A, rows=1), INVALID), (dict(y=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(post=ODD), ALIGN), (dict(gate=ODD, rows=1), ALIGN), (dict(s=None), INVALID), (dict(s=ODD), ALIGN),
]


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(x=None), INVALID), (dict(x=ODD), ALIGN), (dict(sdt=F32, x=HALF), ALIGN), (dict(out=None), INVALID),
    (dict(out=ODD), ALIGN), (dict(m=0, x=None, y=None, post=None, w=None), OK), (dict(d=0, x=None, y=None), OK)])
def test_qblock_norm(kw, status):
    refused(norm(**kw), status)


def norm_backward(s=A, ds=A, sdt=BF16, m=6, d=100, da=A, y=A, dt=BF16, w=A, post=A, gate=None, rows=0, scale=1.0,
                  offset=0.0, eps=1e-6, dx=A, dy=A, dw=A, dp=A, dg=None, ws=A, nws=1 << 40):
    return qp.lib().qblock_norm_backward(s, ds, sdt, m, d, da, y, dt, w, post, gate, rows, scale, offset, eps, dx, dy,
                                         dw, dp, dg, ws, nws, None)


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(ds=ODD), ALIGN), (dict(da=None), INVALID), (dict(da=ODD), ALIGN), (dict(dx=None), INVALID),
    (dict(dx=ODD), ALIGN), (dict(dy=None), INVALID), (dict(dy=ODD), ALIGN), (dict(dw=None), INVALID),
    (dict(dp=None), INVALID), (dict(gate=A, rows=3, dg=None), INVALID), (dict(gate=A, rows=3, dg=ODD), ALIGN),
    (dict(ws=None), INVALID), (dict(nws=100), WORKSPACE), (dict(ws=P(0x10008)), ALIGN),
    (dict(d=0, s=None, dx=None, ws=None), OK)])
def test_qblock_norm_backward(kw, status):
    refused(norm_backward(**kw), status)


def test_workspace_sizes():
    assert qp.qcross_entropy_workspace_bytes(3, 128, 1000, 4, 64, torch.bfloat16) > 0
    assert qp.qcross_entropy_backward_workspace_bytes(3, 128, 1000, 4, 64, torch.bfloat16) > 0
    for bad in ((-1, 128, 40, 4, 64), (3, 96, 40, 4, 64), (3, 128, 40, 5, 64), (3, 128, -1, 4, 64)):
        assert qp.qcross_entropy_workspace_bytes(*bad, torch.float32) == 0
        assert qp.qcross_entropy_backward_workspace_bytes(*bad, torch.float32) == 0
    assert qp.qblock_norm_backward_workspace_bytes(6, 100, 0) >= 3 * 100 * 4
    assert qp.qblock_norm_backward_workspace_bytes(6, 100, 4) == 0
    assert qp.qblock_norm_backward_workspace_bytes(6, 20000, 0) == 0
    # What is kept beside the inputs does not grow with the vocabulary as the logits do.
    rows, k = 4096, 4096
    for v in (128 << 10, 512 << 10):
        grad = qp.qcross_entropy_backward_workspace_bytes(rows, k, v, 4, 64, torch.bfloat16)
        assert grad < rows * v * 2, (grad, rows * v * 2)


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = (torch.zeros((256, 16), dtype=torch.int32), torch.zeros((256, 2), dtype=torch.bfloat16),
         torch.zeros((256, 2), dtype=torch.bfloat16))
    t, f = torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError):
        qp.qcross_entropy(x, t, *w, 4, 64)
    with pytest.raises(ValueError):
        qp.qcross_entropy_backward(x, t, f, f, *w, 4, 64)
    with pytest.raises(ValueError):
        qp.qblock_norm(x, weight=x[0])
    with pytest.raises(ValueError):
        qp.qblock_norm_backward(x, x, weight=x[0])
