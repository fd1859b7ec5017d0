"""The loss and the norms stay inside what they are given: workspaces of exactly the size that
was asked for and outputs of exactly theirs, with marked bytes before and behind; nothing of a
workspace is read that the call has not written (one filled with NaN gives the same bits as
one of zeros); and the backward pass of the norms in place, as include/qpack.h allows it."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, TORCH_DT, dev, log
from test_gpu_loss import case
from test_gpu_norm import Case

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


class Room:
    """Buffers of exact sizes between marked bytes."""

    def __init__(self):
        self.all = []

    def __call__(self, nbytes, fill):
        flat = torch.full((nbytes + 2 * GUARD,), 0x5A, dtype=torch.uint8, device=dev())
        flat[GUARD:GUARD + nbytes] = fill
        self.all.append((flat, nbytes))
        return flat[GUARD:GUARD + nbytes]

    def tensor(self, shape, dtype, fill=0xFF):
        n = torch.empty(shape, dtype=dtype, device="meta").numel()
        return self(n * dtype.itemsize, fill).view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for flat, n in self.all:
            assert (flat[:GUARD] == 0x5A).all() and (flat[GUARD + n:] == 0x5A).all()


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,k,v,bits,gs", [
    (1, 64, 5, 4, 32), (2, 4096, 300, 4, 64), (3, 32, 4099, 8, 32), (16, 96, 66001, 2, 32), (17, 288, 65, 6, 32),
    (33, 8256, 259, 3, 32), (70, 256, 700, 4, 64), (129, 384, 1001, 8, 128), (300, 768, 33001, 4, 64), (40, 32, 4097, 4, 32),
    (5000, 32, 12500, 4, 32), (16500, 64, 4100, 3, 64)])
def test_loss(m, k, v, bits, gs, dt):
    log(f"room of the loss: m={m} k={k} v={v} bits={bits} gs={gs} dt={dt}")
    x, w, t, dloss = case(m, k, v, bits, gs, dt)
    x, t, dloss, w, T = x.to(dev()), t.to(dev()), dloss.to(dev()), oh.cuda(w), TORCH_DT[dt]
    stream = torch.cuda.current_stream().cuda_stream
    runs = []
    for fill in (0, 0xFF):
        room = Room()
        loss, lse = (room.tensor((m,), torch.float32) for _ in range(2))
        dx, ds, db = room.tensor((m, k), T), room.tensor((v, k // gs), T), room.tensor((v, k // gs), T)
        n = qp.qcross_entropy_workspace_bytes(m, k, v, bits, gs, T)
        ws = room(n, fill)
        head = (*(p.data_ptr() for p in w), dt, v, bits, gs)
        qp.check(qp.lib().qcross_entropy(ptr(x), dt, m, k, ptr(t), *head, ptr(loss), ptr(lse), ptr(ws), n, stream))
        n = qp.qcross_entropy_backward_workspace_bytes(m, k, v, bits, gs, T)
        ws = room(n, fill)
        qp.check(qp.lib().qcross_entropy_backward(ptr(x), dt, m, k, ptr(t), ptr(lse), ptr(dloss), *head, ptr(dx), ptr(ds),
                                                  ptr(db), ptr(ws), n, stream))
        room.check()
        runs.append((loss, lse, dx, ds, db))
    assert all(oh.same_bits(a, b) and a.isfinite().all() for a, b in zip(*runs))


NORMS = [(1, 7, 1), (5, 96, 5), (9, 1027, 3), (40, 1500, 1), (77, 2881, 0), (12, 5120, 4), (1030, 136, 515), (600, 8300, 600),
         (700, 8200, 1), (7, 16384, 0)]


@pytest.mark.parametrize("dt,sdt", [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("m,d,gates", NORMS)
def test_norms(m, d, gates, dt, sdt):
    log(f"room of the norms: m={m} d={d} gates={gates} dt={dt} sdt={sdt}")
    c = Case(m, d, dt, sdt, True, gates, True)
    p, T, S = c.parts(), TORCH_DT[dt], TORCH_DT[sdt]
    x, da, ds = c.x.to(dev()), c.da.to(dev()), c.ds.to(dev())
    stream = torch.cuda.current_stream().cuda_stream
    weights = (ptr(p["weight"]), ptr(p["post_weight"]), ptr(p["gate"]), gates, c.factor, c.offset, 1e-5)
    n = qp.qblock_norm_backward_workspace_bytes(m, d, gates)
    runs = []
    for fill in (0, 0xFF):
        room = Room()
        s, a = room.tensor((m, d), S), room.tensor((m, d), T)
        qp.check(qp.lib().qblock_norm(ptr(x), sdt, m, d, ptr(p["y"]), dt, *weights, ptr(s), ptr(a), stream))
        dx, dy, dw, dp = room.tensor((m, d), S), room.tensor((m, d), T), room.tensor((d,), T), room.tensor((d,), T)
        dg = room.tensor((gates, d), T) if gates else None
        ws = room(n, fill)
        qp.check(qp.lib().qblock_norm_backward(ptr(s), ptr(ds), sdt, m, d, ptr(da), ptr(p["y"]), dt, *weights, ptr(dx), ptr(dy),
                                               ptr(dw), ptr(dp), ptr(dg), ptr(ws), n, stream))
        room.check()
        runs.append([s, a, dx, dy, dw, dp] + ([dg] if gates else []))
    assert all(oh.same_bits(a, b) and a.isfinite().all() for a, b in zip(*runs))
    # dx over ds; dy over da, and over y.
    want = runs[0]
    for over in ("da", "y"):
        out = {"ds": ds.clone(), "da": da.clone(), "y": p["y"].clone()}
        dw, dp = torch.empty_like(p["weight"]), torch.empty_like(p["post_weight"])
        dg = torch.empty_like(p["gate"]) if gates else None
        ws = torch.empty(n, dtype=torch.uint8, device=dev())
        qp.check(qp.lib().qblock_norm_backward(
            ptr(want[0]), ptr(out["ds"]), sdt, m, d, ptr(out["da"]), ptr(out["y"]), dt, *weights, ptr(out["ds"]), ptr(out[over]),
            ptr(dw), ptr(dp), ptr(dg), ptr(ws), n, stream))
        torch.cuda.synchronize()
        got = [out["ds"], out[over], dw, dp] + ([dg] if gates else [])
        assert all(oh.same_bits(a, b) for a, b in zip(want[2:], got)), over


@pytest.mark.parametrize("post,pre,y", [(False, True, True), (True, False, True), (False, False, True), (False, True, False)])
@pytest.mark.parametrize("m,d", [(20, 700), (30, 6000), (600, 8300)])
def test_norms_in_place_with_parts_left_out(m, d, post, pre, y):
    c = Case(m, d, BF16, BF16, post, 0, pre, y=y)
    p, ds = c.parts(), c.ds.to(dev())
    da = c.da.to(dev()) if pre else None
    s = c.x.to(dev())
    want = qp.qblock_norm_backward(s, da, ds, **p)
    n = qp.qblock_norm_backward_workspace_bytes(m, d, 0)
    stream = torch.cuda.current_stream().cuda_stream
    for over in (["da"] if pre and y else []) + (["y"] if y else ["none"]):
        out = {"ds": ds.clone(), "da": None if da is None else da.clone(), "y": p["y"].clone() if y else None, "none": None}
        dw, dp = (None if t is None else torch.empty_like(t) for t in (p["weight"], p["post_weight"]))
        ws = torch.empty(n, dtype=torch.uint8, device=dev())
        qp.check(qp.lib().qblock_norm_backward(
            ptr(s), ptr(out["ds"]), BF16, m, d, ptr(out["da"]), ptr(out["y"]), BF16, ptr(p["weight"]), ptr(p["post_weight"]), None,
            0, c.factor, c.offset, 1e-5, ptr(out["ds"]), ptr(out[over]), ptr(dw), ptr(dp), None, ptr(ws), n, stream))
        torch.cuda.synchronize()
        assert oh.same_bits(out["ds"], want[0]) and (not y or oh.same_bits(out[over], want[1])), over
        assert all(a is None or oh.same_bits(a, b) for a, b in ((dw, want[2]), (dp, want[3])))
