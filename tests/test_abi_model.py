"""Host-side checks of the operators around the products (no GPU needed): every
argument error is reported with its status and a message before any HIP call,
calls with nothing to do succeed, and workspace sizes are 0 for what is
refused."""
from __future__ import annotations

import ctypes

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp

OK, INVALID, UNSUPPORTED, MISMATCH, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5, 6
F32, F16, BF16 = qp.QP_F32, qp.QP_F16, qp.QP_BF16
P = ctypes.c_void_p
A = P(0x10000)      # a well-aligned stand-in address (never dereferenced)
ODD = P(0x10001)    # misaligned for every element size
LAYOUT = [
    (dict(bits=5), UNSUPPORTED), (dict(bits=0), UNSUPPORTED), (dict(gs=16), UNSUPPORTED),
    (dict(gs=0), UNSUPPORTED), (dict(gs=-32), UNSUPPORTED),
]
BIG = 1 << 40


def refused(status, want):
    assert status == want, (status, qp.last_error())
    if want != OK:
        assert qp.last_error()


def ffn(x=A, dt=BF16, m=2, d=128, f=256, gate=(A, A, A), up=(A, A, A), down=(A, A, A), sdt=None, bits=4,
        gs=64, act=0, saved=None, y=A, ws=A, nws=1 << 30):
    return qp.lib().qffn(x, dt, m, d, f, *gate, *up, *down, dt if sdt is None else sdt, bits, gs, act, saved,
                         y, ws, nws, None)


FFN = LAYOUT + [
    (dict(d=96), SHAPE), (dict(f=96), SHAPE), (dict(m=-1), INVALID), (dict(d=-64), INVALID), (dict(f=-64), INVALID),
    (dict(dt=7), INVALID), (dict(sdt=F16), MISMATCH), (dict(act=2), UNSUPPORTED), (dict(act=-1), UNSUPPORTED),
    (dict(m=BIG), INVALID), (dict(d=BIG), INVALID), (dict(f=BIG), INVALID),
    (dict(gate=(None, A, A)), INVALID), (dict(up=(A, None, A)), INVALID), (dict(down=(A, A, None)), INVALID),
    (dict(gate=(P(0x10002), A, A)), ALIGN), (dict(up=(A, ODD, A)), ALIGN), (dict(down=(A, A, ODD)), ALIGN),
    (dict(x=None), INVALID), (dict(x=ODD), ALIGN), (dict(saved=ODD), ALIGN),
]


@pytest.mark.parametrize("kw,status", FFN + [
    (dict(y=None), INVALID), (dict(y=ODD), ALIGN), (dict(ws=None), INVALID), (dict(nws=15), WORKSPACE),
    (dict(ws=P(0x10008)), ALIGN), (dict(m=0, x=None, y=None, ws=None), OK)])
def test_qffn(kw, status):
    refused(ffn(**kw), status)


def ffn_backward(x=A, dy=A, saved=A, dt=BF16, m=2, d=128, f=256, gate=(A, A, A), up=(A, A, A), down=(A, A, A),
                 sdt=None, bits=4, gs=64, act=0, dx=A, grads=(A,) * 6, ws=A, nws=1 << 30):
    return qp.lib().qffn_backward(x, dy, saved, dt, m, d, f, *gate, *up, *down, dt if sdt is None else sdt, bits,
                                  gs, act, dx, *grads, ws, nws, None)


@pytest.mark.parametrize("kw,status", FFN + [
    (dict(saved=None), INVALID), (dict(dy=None), INVALID), (dict(dy=ODD), ALIGN), (dict(dx=ODD), ALIGN),
    (dict(grads=(A, None, A, A, A, A)), INVALID), (dict(grads=(A, A, None, A, A, A)), INVALID),
    (dict(grads=(A, A, A, A, A, ODD)), ALIGN), (dict(ws=None), INVALID), (dict(nws=64), WORKSPACE),
    (dict(ws=P(0x10004)), ALIGN), (dict(dx=None, grads=(None,) * 6, x=None, dy=None, ws=None), OK)])
def test_qffn_backward(kw, status):
    refused(ffn_backward(**kw), status)


def linear(x=A, dy=A, dt=BF16, m=2, k=128, w=(A, A, A), sdt=None, n=40, bits=4, gs=64, dx=A, ds=A, db=A, ws=A,
           nws=1 << 30):
    return qp.lib().qmatmul_backward(x, dy, dt, m, k, *w, dt if sdt is None else sdt, n, bits, gs, dx, ds, db, ws,
                                     nws, None)


@pytest.mark.parametrize("kw,status", LAYOUT + [
    (dict(k=96), SHAPE), (dict(m=-1), INVALID), (dict(k=-64), INVALID), (dict(n=-1), INVALID),
    (dict(m=BIG), INVALID), (dict(n=BIG), INVALID), (dict(dt=3), INVALID), (dict(sdt=F32), MISMATCH),
    (dict(x=None), INVALID), (dict(x=ODD), ALIGN), (dict(dy=None), INVALID), (dict(dy=ODD), ALIGN),
    (dict(w=(None, A, A)), INVALID), (dict(w=(A, None, A)), INVALID), (dict(w=(A, A, ODD)), ALIGN),
    (dict(ds=None), INVALID), (dict(db=None), INVALID), (dict(dx=ODD), ALIGN), (dict(ds=ODD), ALIGN),
    (dict(n=41, ws=None), INVALID), (dict(n=41, nws=8), WORKSPACE), (dict(n=41, ws=ODD), ALIGN),
    (dict(dx=None, ds=None, db=None, x=None, dy=None), OK)])
def test_qmatmul_backward(kw, status):
    refused(linear(**kw), status)


def embedding(ids=A, t=3, w=(A, A, A), dt=BF16, v=40, k=128, bits=4, gs=64, factor=1.0, out=A):
    return qp.lib().qembedding(ids, t, *w, dt, v, k, bits, gs, factor, out, None)


@pytest.mark.parametrize("kw,status", LAYOUT + [
    (dict(k=96), SHAPE), (dict(t=-1), INVALID), (dict(v=-1), INVALID), (dict(k=-64), INVALID), (dict(dt=3), INVALID),
    (dict(t=BIG), INVALID), (dict(v=(1 << 31) - 1), INVALID), (dict(ids=None), INVALID), (dict(ids=P(0x10002)), ALIGN),
    (dict(out=None), INVALID), (dict(out=ODD), ALIGN), (dict(w=(A, A, None)), INVALID), (dict(w=(ODD, A, A)), ALIGN),
    (dict(t=0, ids=None, out=None), OK), (dict(k=0, ids=None, out=None), OK)])
def test_qembedding(kw, status):
    refused(embedding(**kw), status)


def embedding_backward(ids=A, t=3, dout=A, dt=BF16, wq=A, v=40, k=128, bits=4, gs=64, factor=1.0, ds=A, db=A, ws=A,
                       nws=1 << 30):
    return qp.lib().qembedding_backward(ids, t, dout, dt, wq, v, k, bits, gs, factor, ds, db, ws, nws, None)


@pytest.mark.parametrize("kw,status", LAYOUT + [
    (dict(k=96), SHAPE), (dict(t=-1), INVALID), (dict(v=-1), INVALID), (dict(dt=-1), INVALID), (dict(t=BIG), INVALID),
    (dict(ids=None), INVALID), (dict(dout=None), INVALID), (dict(dout=ODD), ALIGN), (dict(wq=None), INVALID),
    (dict(wq=P(0x10002)), ALIGN), (dict(ds=None), INVALID), (dict(db=ODD), ALIGN), (dict(ws=None), INVALID),
    (dict(nws=4), WORKSPACE), (dict(ws=P(0x10008)), ALIGN), (dict(v=0, ids=None, ds=None), OK)])
def test_qembedding_backward(kw, status):
    refused(embedding_backward(**kw), status)


def logits(x=A, dt=BF16, rows=2, v=100, istride=100, hist=A, nhist=5, offs=A, plens=None, rep=A, freq=None,
           pres=None, bids=None, bvals=None, nbias=0, boffs=None, mask=None, mstride=0, out=A, ostride=100):
    return qp.lib().qlogits_adjust(x, dt, rows, v, istride, hist, nhist, offs, plens, rep, freq, pres, bids, bvals,
                                   nbias, boffs, mask, mstride, out, ostride, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(v=-1), INVALID), (dict(nhist=-1), INVALID), (dict(nbias=-1), INVALID),
    (dict(dt=5), INVALID), (dict(rows=BIG), INVALID), (dict(v=BIG), INVALID), (dict(istride=99), SHAPE),
    (dict(ostride=99), SHAPE), (dict(mask=A, mstride=3), SHAPE), (dict(x=None), INVALID), (dict(x=ODD), ALIGN),
    (dict(out=None), INVALID), (dict(out=ODD), ALIGN), (dict(hist=None, offs=None), INVALID),
    (dict(hist=None), INVALID), (dict(offs=None, rep=None), INVALID), (dict(nbias=2, boffs=A), INVALID),
    (dict(nbias=2, bids=A, bvals=A), INVALID), (dict(rep=P(0x10002)), ALIGN), (dict(hist=ODD), ALIGN),
    (dict(mask=ODD, mstride=4), ALIGN), (dict(rows=0, x=None, out=None), OK), (dict(v=0, x=None, out=None), OK)])
def test_qlogits_adjust(kw, status):
    refused(logits(**kw), status)


def test_workspace_sizes():
    assert qp.qffn_workspace_bytes(3, 128, 256, torch.bfloat16) >= 3 * 256 * 2
    assert qp.qffn_workspace_bytes(-1, 128, 256, torch.bfloat16) == 0
    assert qp.qffn_backward_workspace_bytes(3, 128, 256, 4, 64, torch.float32) >= 3 * 3 * 256 * 4
    for bad in ((-1, 128, 256, 4, 64), (3, 96, 256, 4, 64), (3, 128, 256, 5, 64), (3, 128, 256, 4, 48)):
        assert qp.qffn_backward_workspace_bytes(*bad, torch.float32) == 0
    assert qp.qmatmul_backward_workspace_bytes(5, 128, 41, 4, 64, torch.float16) >= 5 * 48 * 2   # padded dy
    assert qp.qmatmul_backward_workspace_bytes(5, 128, -1, 4, 64, torch.float16) == 0
    assert qp.qembedding_backward_workspace_bytes(100, 128, 4, 64) >= 100 * 4
    assert qp.qembedding_backward_workspace_bytes(100, 100, 4, 32) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = (torch.zeros((256, 16), dtype=torch.int32), torch.zeros((256, 2), dtype=torch.bfloat16),
         torch.zeros((256, 2), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qp.qffn(x, w, w, w, 4, 64)
    with pytest.raises(ValueError):
        qp.qmatmul_backward(x, x, *w, 4, 64)
    with pytest.raises(ValueError):
        qp.qembedding(torch.zeros(3, dtype=torch.int32), *w, 4, 64)
    with pytest.raises(ValueError):
        qp.qlogits_adjust(x)
    with pytest.raises(ValueError):
        qp._act_code("relu")
