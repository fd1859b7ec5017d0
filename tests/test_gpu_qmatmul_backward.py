"""GPU parity of qmatmul_backward with its 64-bit form, and with differences.

Bounds (ophelpers): dx: TAU * S + half an ulp with S = |dy| |W|; dscales and
dbiases: the operands dy, x and q are exact, so only fp32 sums over the rows and
the group round: gamma(m + gs) * (|dy|^T |x| weighted like the sum) + half an ulp.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, TAU, dev, log

pytestmark = pytest.mark.gpu


def reference(x, dy, w, bits, gs, dt):
    W = oh.dense(w, bits, gs)
    xd, dyd = x.double(), dy.double()
    dx = dyd @ W
    b_dx = TAU[dt] * (dyd.abs() @ W.abs()) + oh.half_ulp(dx, dt)
    ds, db = oh.group_sums(w, dyd.t() @ xd, bits, gs)
    S = oh.group_sums(w, dyd.abs().t() @ xd.abs(), bits, gs)
    g = oh.gamma(x.shape[0] + gs)
    return [(dx, b_dx), (ds, g * S[0] + oh.half_ulp(ds, dt)), (db, g * S[1] + oh.half_ulp(db, dt))]


def case(m, k, n, bits, gs, dt):
    g = oh.rng(oh.seed_of(m, k, n, bits, gs, dt))
    return (oh.normal((m, k), 1.0, dt, g), oh.normal((m, n), 0.5, dt, g),
            oh.weight(n, k, bits, gs, dt, g))


def run_and_check(m, k, n, bits, gs, dt, what=""):
    x, dy, w = case(m, k, n, bits, gs, dt)
    log(f"qmatmul_backward {what}: m={m} k={k} n={n} bits={bits} gs={gs} dt={dt}")
    out = qp.qmatmul_backward(x.to(dev()), dy.to(dev()), *oh.cuda(w), bits, gs)
    torch.cuda.synchronize()
    for y, (ref, bound), name in zip(out, reference(x, dy, w, bits, gs, dt), ("dx", "ds", "db")):
        oh.check(y, ref, bound, f"{what} {name}")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (4, 32), (6, 32), (8, 32), (2, 64), (3, 64),
                                     (4, 64), (6, 64), (8, 64), (4, 128), (3, 128), (6, 128)])
def test_every_width_and_group(bits, gs, dt):
    run_and_check(75, 384, 200, bits, gs, dt, "widths")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,k,n", [
    (1, 32, 1), (1, 128, 40), (2, 96, 7), (3, 160, 33), (16, 64, 64), (17, 288, 65), (31, 256, 8),
    (33, 512, 1000), (64, 64, 129), (65, 1056, 31), (127, 128, 255), (129, 256, 256), (200, 544, 513),
    (256, 256, 256), (257, 320, 264), (300, 768, 1001), (515, 288, 90),
])
def test_odd_and_whole_sizes(m, k, n, dt):
    run_and_check(m, k, n, 4, 32, dt, "sizes")


@pytest.mark.parametrize("bits", [2, 4, 8])
def test_long_contraction_and_many_rows(bits):
    run_and_check(1100, 512, 96, bits, 64, BF16, "many rows")
    run_and_check(20, 256, 8200, bits, 64, F16, "long contraction")


@pytest.mark.parametrize("m,k,n,bits,gs,dt", [
    (1, 4096, 4096, 4, 64, BF16), (65, 4128, 4010, 4, 32, F16), (140, 4096, 4104, 8, 128, BF16),
    (257, 2048, 8201, 2, 64, BF16), (64, 4224, 4096, 3, 32, F16), (200, 8192, 2050, 6, 64, BF16)])
def test_weights_of_many_tiles(m, k, n, bits, gs, dt):
    """Weights large enough for the persistent tiles, ragged in every direction."""
    run_and_check(m, k, n, bits, gs, dt, "many tiles")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("m,k,n", [(70, 256, 96), (300, 512, 264)])
def test_misaligned_bases(m, k, n, dt):
    """Views one element into their storage: element alignment is all that is asked for."""
    x, dy, w = case(m, k, n, 4, 32, dt)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:] = t.flatten().to(dev())
        return flat[1:].view(t.shape)

    wq, s, b = w
    out = qp.qmatmul_backward(shifted(x), shifted(dy), shifted(wq), shifted(s), shifted(b), 4, 32)
    torch.cuda.synchronize()
    for y, (ref, bound), name in zip(out, reference(x, dy, w, 4, 32, dt), ("dx", "ds", "db")):
        oh.check(y, ref, bound, f"misaligned {name}")


def test_deterministic_and_parts_agree():
    x, dy, w = case(130, 512, 700, 4, 64, BF16)
    args = (x.to(dev()), dy.to(dev()), *oh.cuda(w), 4, 64)
    a, b = qp.qmatmul_backward(*args), qp.qmatmul_backward(*args)
    only_x = qp.qmatmul_backward(*args, weight_grads=False)
    only_w = qp.qmatmul_backward(*args, input_grad=False)
    torch.cuda.synchronize()
    assert all(oh.same_bits(p, q) for p, q in zip(a, b))
    assert only_x[1] is None and only_x[2] is None and oh.same_bits(only_x[0], a[0])
    assert only_w[0] is None and oh.same_bits(only_w[1], a[1]) and oh.same_bits(only_w[2], a[2])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_empty_rows_and_columns(dt):
    x, dy, w = case(4, 64, 40, 4, 32, dt)
    wd = oh.cuda(w)
    dx, ds, db = qp.qmatmul_backward(x[:0].to(dev()), dy[:0].to(dev()), *wd, 4, 32)
    assert dx.shape == (0, 64) and not ds.any() and not db.any()
    dx, ds, db = qp.qmatmul_backward(x.to(dev()), dy[:, :0].contiguous().to(dev()),
                                     *(t[:0] for t in wd), 4, 32)
    assert not dx.any() and ds.shape == (0, 2)


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("m,k,n", [(66, 256, 264), (300, 512, 264)])
def test_infinity_and_nan_stay_in_their_rows(m, k, n, dt):
    """A row of dy with an infinity or a NaN spoils its own row of dx and the
    weight rows it meets, nothing else (in particular not across a padded edge)."""
    x, dy, w = case(m, k, n, 4, 32, dt)
    ref = qp.qmatmul_backward(x.to(dev()), dy.to(dev()), *oh.cuda(w), 4, 32)
    dy2 = dy.clone()
    dy2[m - 1, n - 1] = float("nan")
    out = qp.qmatmul_backward(x.to(dev()), dy2.to(dev()), *oh.cuda(w), 4, 32)
    torch.cuda.synchronize()
    assert oh.same_bits(out[0][:-1], ref[0][:-1]) and out[0][-1].isnan().all()
    for i in (1, 2):
        assert oh.same_bits(out[i][:-1], ref[i][:-1]) and out[i][-1].isnan().all()


@pytest.mark.parametrize("bits,gs", [(3, 32), (4, 64)])
def test_against_differences(bits, gs):
    """<grad, direction> against central differences of the 64-bit forward pass
    (bilinear in x and in the scales and biases: the differences are exact up to
    their own rounding, below 1e-9 of the sum of magnitudes)."""
    m, k, n = 21, 192, 50
    x, dy, w = case(m, k, n, bits, gs, F32)
    out = qp.qmatmul_backward(x.to(dev()), dy.to(dev()), *oh.cuda(w), bits, gs)
    g = oh.rng(5)
    dirs = [torch.randn(t.shape, generator=g).double() for t in (x, w[1], w[2])]
    q = oh.codes(w[0], bits)

    def loss(xx, ss, bb):
        W = q * ss.repeat_interleave(gs, 1) + bb.repeat_interleave(gs, 1)
        return float((dy.double() * (xx @ W.t())).sum())

    base = [x.double(), w[1].double(), w[2].double()]
    eps = 1e-4
    mag = float((dy.double().abs() * (x.double().abs() @ oh.dense(w, bits, gs).abs().t())).sum())
    for i, (ref, bound) in enumerate(reference(x, dy, w, bits, gs, F32)):
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + eps * dirs[i], base[i] - eps * dirs[i]
        fd = (loss(*up) - loss(*down)) / (2 * eps)
        got = float((out[i].cpu().double() * dirs[i]).sum())
        assert abs(got - fd) <= float((bound * dirs[i].abs()).sum()) + 1e-9 * mag / eps, (i, got, fd)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("m,k,n", [(70, 256, 96), (130, 512, 265), (300, 512, 264), (33, 4096, 4160)])
def test_alignment_changes_nothing(m, k, n, dt):
    """One kernel for a shape: the same bits wherever the operands lie, all of them off
    16-byte addresses or one alone (the input gradient does not read x at all)."""
    x, dy, w = case(m, k, n, 4, 32, dt)
    wd = oh.cuda(w)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:] = t.flatten().to(dev())
        return flat[1:].view(t.shape)

    xd, dyd = x.to(dev()), dy.to(dev())
    want = qp.qmatmul_backward(xd, dyd, *wd, 4, 32)
    log(f"qmatmul_backward at other addresses: m={m} k={k} n={n} dt={dt}")
    for xx, yy, ww in ((shifted(x), dyd, wd), (xd, shifted(dy), wd),
                       (shifted(x), shifted(dy), tuple(shifted(t) for t in wd))):
        got = qp.qmatmul_backward(xx, yy, *ww, 4, 32)
        only_x = qp.qmatmul_backward(xx, yy, *ww, 4, 32, weight_grads=False)
        torch.cuda.synchronize()
        assert all(oh.same_bits(a, b) for a, b in zip(got, want)) and oh.same_bits(only_x[0], want[0])
