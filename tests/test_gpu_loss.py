"""GPU parity of qcross_entropy and its backward pass with their 64-bit forms, and with
differences of the loss.

Bounds, with S = |x| (q |s| + |b|)^T the magnitudes that a logit's sum is made of (the
product folds the scales out of the codes' sums) and G the groups of a row:
* a logit: (k + 2 G + 64) 2^-24 S for the fp32 sums, and 2^-17 S where the groups' sums of
  x are operands of 16 bits, in two parts;
* lse: the largest of its logits' bounds, and the roundings of exp, of sums that are
  never longer than some hundreds in a row, and of log: 2^-16 + 2^-22 |lse|; the loss: that
  and its target's logit;
* dz = g (p - [target]): |g| p (bound of z + 2^-20 (1 + |z - lse|)), |g| 2^-126 (the exponential
  instruction gives 0 where its result would be below fp32's normal range) + half an ulp of the
  products' operand (of 16 bits: times a factor that makes the largest |g| 2^14, and three
  roundings of 2^-24 for the factor);
* dx: that of dz times |W|, TAU |dz| |W| and half an ulp; dscales and dbiases: that of dz
  times |x|, summed as they are, fp32 sums over the rows and the group, half an ulp.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, HALF_SUBNORMAL, HALF_ULP, TAU, dev, log

pytestmark = pytest.mark.gpu


def case(m, k, v, bits, gs, dt, sigma=2.0):
    g = oh.rng(oh.seed_of(m, k, v, bits, gs, dt))
    x = oh.normal((m, k), sigma, dt, g)
    w = oh.weight(v, k, bits, gs, dt, g)
    t = torch.randint(0, max(v, 1), (m,), generator=g).to(torch.int32)
    if m > 2:
        t[1], t[m - 1] = -100, v      # no target
    dloss = torch.rand(m, generator=g) / m + 0.1 / m
    return x, w, t, dloss


def logits64(x, w, bits, gs, dt):
    wq, s, b = w
    xd = x.double()
    W = oh.dense(w, bits, gs)
    mags = oh.codes(wq, bits) * oh.spread(s, gs).abs() + oh.spread(b, gs).abs()
    S = xd.abs() @ mags.t()
    k = x.shape[1]
    per = (k + 2 * (k // gs) + 64) * 2.0 ** -24 + (2.0 ** -17 if dt != F32 else 0.0)
    return xd @ W.t(), per * S, W


def forward64(x, w, t, bits, gs, dt):
    z, bz, W = logits64(x, w, bits, gs, dt)
    lse = torch.logsumexp(z, 1)
    b_lse = bz.max(1).values + 2.0 ** -16 + 2.0 ** -22 * lse.abs()
    live = (t >= 0) & (t < w[0].shape[0])
    at = torch.where(live, t.long(), 0)[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
    b_loss = torch.where(live, b_lse + bz.gather(1, at)[:, 0] + 2.0 ** -23 * (loss.abs() + lse.abs()), 0.0)
    return (loss, b_loss), (lse, b_lse), (z, bz, W, live, at)


def backward64(x, w, t, lse, dloss, bits, gs, dt):
    """(ref, bound) of dx, dscales, dbiases at the lse that was given."""
    _, _, (z, bz, W, live, at) = forward64(x, w, t, bits, gs, dt)
    g = torch.where(live, dloss.double(), 0.0)[:, None]
    off = z - lse.double()[:, None]
    p = torch.exp(off)
    dz = p.clone()
    dz.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    dz = dz * g
    floor = HALF_SUBNORMAL[dt] * (float(g.abs().max()) * 2.0 ** -14 if dt == F16 else 1.0)
    b_dz = g.abs() * p * (1.01 * bz + 2.0 ** -20 * (1 + off.abs())) + dz.abs() * 2.0 ** -22 + g.abs() * 2.0 ** -126
    b_dz = b_dz + torch.clamp(1.01 * dz.abs() * HALF_ULP[dt], min=floor)
    b_dz = torch.where(live[:, None], b_dz, 0.0)
    xd = x.double()
    dx = dz @ W
    b_dx = b_dz @ W.abs() + TAU[dt] * (dz.abs() @ W.abs()) + oh.half_ulp(dx, dt)
    out = [(dx, b_dx)]
    refs = oh.group_sums(w, dz.t() @ xd, bits, gs)
    err = oh.group_sums(w, b_dz.t() @ xd.abs(), bits, gs)
    mags = oh.group_sums(w, dz.abs().t() @ xd.abs(), bits, gs)
    gam = oh.gamma(x.shape[0] + gs)
    return out + [(r, 1.01 * e + gam * s + oh.half_ulp(r, dt)) for r, e, s in zip(refs, err, mags)]


def run_and_check(m, k, v, bits, gs, dt, what, sigma=2.0, move=lambda t: t.to(dev())):
    x, w, t, dloss = case(m, k, v, bits, gs, dt, sigma)
    log(f"qcross_entropy {what}: m={m} k={k} v={v} bits={bits} gs={gs} dt={dt}")
    xd, td, wd = move(x), move(t), tuple(move(p) for p in w)
    loss, lse = qp.qcross_entropy(xd, td, *wd, bits, gs)
    torch.cuda.synchronize()
    (r_loss, b_loss), (r_lse, b_lse), _ = forward64(x, w, t, bits, gs, dt)
    oh.check(lse, r_lse, b_lse, f"{what} lse")
    oh.check(loss, r_loss, b_loss, f"{what} loss")
    log(f"qcross_entropy_backward {what}")
    grads = qp.qcross_entropy_backward(xd, td, lse, move(dloss), *wd, bits, gs)
    torch.cuda.synchronize()
    for got, (ref, bound), name in zip(grads, backward64(x, w, t, lse.cpu(), dloss, bits, gs, dt), ("dx", "ds", "db")):
        oh.check(got, ref, bound, f"{what} {name}")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m", [5, 75])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (4, 32), (6, 32), (8, 32), (2, 64), (3, 64), (4, 64), (6, 64),
                                     (8, 64), (2, 128), (3, 128), (4, 128), (6, 128), (8, 128)])
def test_every_width_and_group(bits, gs, m, dt):
    run_and_check(m, 384, 700, bits, gs, dt, "widths")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,k,v", [
    (1, 32, 1), (1, 128, 40), (2, 96, 7), (3, 160, 33), (16, 64, 64), (17, 32, 300), (17, 288, 65), (33, 96, 1000),
    (64, 64, 129), (65, 1056, 31), (127, 128, 255), (128, 256, 256), (129, 256, 257), (200, 544, 513), (257, 320, 264),
    (300, 768, 1001), (40, 128, 4096), (40, 128, 4097), (7, 64, 9001)])
def test_odd_and_whole_sizes(m, k, v, dt):
    run_and_check(m, k, v, 4, 32, dt, "sizes")


@pytest.mark.parametrize("m,k,v,bits,gs,dt", [
    (1, 4096, 5000, 4, 64, BF16), (12, 2048, 6001, 8, 32, F16), (16, 4096, 2050, 3, 128, BF16),
    (77, 1024, 9001, 6, 32, F16), (140, 2048, 4104, 2, 64, BF16), (520, 512, 3001, 4, 64, F16)])
def test_larger(m, k, v, bits, gs, dt):
    run_and_check(m, k, v, bits, gs, dt, "larger")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_far_logits(dt):
    """Logits of some hundreds: the maximum is subtracted before any exponential."""
    run_and_check(40, 128, 600, 4, 32, dt, "far", sigma=100.0)


def shifted(t):
    """A copy one element into its storage."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
    flat[1:] = t.flatten().to(dev())
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("m,k,v", [(2, 128, 90), (9, 256, 500), (70, 256, 700)])
def test_misaligned_bases(m, k, v, dt):
    run_and_check(m, k, v, 4, 32, dt, "misaligned", move=shifted)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("m,k,v", [(9, 256, 500), (70, 256, 700), (300, 512, 1030)])
def test_alignment_changes_nothing(m, k, v, dt):
    x, w, t, dloss = case(m, k, v, 4, 32, dt)
    runs = []
    for move in (lambda t: t.to(dev()), shifted):
        xd, td, wd = move(x), move(t), tuple(move(p) for p in w)
        loss, lse = qp.qcross_entropy(xd, td, *wd, 4, 32)
        runs.append((loss, lse, *qp.qcross_entropy_backward(xd, td, lse, move(dloss), *wd, 4, 32)))
    torch.cuda.synchronize()
    assert all(oh.same_bits(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("m", [3, 130])
def test_deterministic_and_parts_agree(m):
    x, w, t, dloss = case(m, 512, 700, 4, 64, BF16)
    xd, td, gd, wd = x.to(dev()), t.to(dev()), dloss.to(dev()), oh.cuda(w)
    (loss, lse), again = qp.qcross_entropy(xd, td, *wd, 4, 64), qp.qcross_entropy(xd, td, *wd, 4, 64)
    args = (xd, td, lse, gd, *wd, 4, 64)
    a, b = qp.qcross_entropy_backward(*args), qp.qcross_entropy_backward(*args)
    only_x = qp.qcross_entropy_backward(*args, weight_grads=False)
    only_w = qp.qcross_entropy_backward(*args, input_grad=False)
    torch.cuda.synchronize()
    assert oh.same_bits(loss, again[0]) and oh.same_bits(lse, again[1])
    assert all(oh.same_bits(p, q) for p, q in zip(a, b))
    assert only_x[1] is None and only_x[2] is None and oh.same_bits(only_x[0], a[0])
    assert only_w[0] is None and oh.same_bits(only_w[1], a[1]) and oh.same_bits(only_w[2], a[2])


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m", [4, 70])
def test_no_target_at_all(m, dt):
    x, w, t, dloss = case(m, 128, 300, 4, 32, dt)
    none = torch.full_like(t, -1).to(dev())
    wd = oh.cuda(w)
    loss, lse = qp.qcross_entropy(x.to(dev()), none, *wd, 4, 32)
    grads = qp.qcross_entropy_backward(x.to(dev()), none, lse, torch.full_like(dloss, float("nan")).to(dev()), *wd, 4, 32)
    torch.cuda.synchronize()
    assert not loss.any() and torch.isfinite(lse).all() and not any(g.any() for g in grads)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m", [4, 70, 300])
def test_nan_stays_in_its_row(m, dt):
    """A row of x with a NaN: its own loss and dx row; all other rows keep their bits."""
    x, w, t, dloss = case(m, 256, 700, 4, 32, dt)
    t[:] = 5
    wd, td, gd = oh.cuda(w), t.to(dev()), dloss.to(dev())
    bad = x.clone()
    bad[m - 1, 255] = float("nan")
    runs = []
    for xx in (x, bad):
        loss, lse = qp.qcross_entropy(xx.to(dev()), td, *wd, 4, 32)
        runs.append((loss, lse, qp.qcross_entropy_backward(xx.to(dev()), td, lse, gd, *wd, 4, 32, weight_grads=False)[0]))
    torch.cuda.synchronize()
    for a, b in zip(*runs):
        assert b[m - 1].isnan().all()
        if dt != F16:
            assert oh.same_bits(a[:m - 1], b[:m - 1])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_empty(dt):
    x, w, t, dloss = case(4, 64, 40, 4, 32, dt)
    xd, td, wd, gd = x.to(dev()), t.to(dev()), oh.cuda(w), dloss.to(dev())
    loss, lse = qp.qcross_entropy(xd[:0], td[:0], *wd, 4, 32)
    dx, ds, db = qp.qcross_entropy_backward(xd[:0], td[:0], lse, gd[:0], *wd, 4, 32)
    assert loss.shape == (0,) and dx.shape == (0, 64) and not ds.any() and not db.any()
    none = tuple(p[:0] for p in wd)
    loss, lse = qp.qcross_entropy(xd, td, *none, 4, 32)
    assert not loss.any() and (lse == float("-inf")).all()
    dx, ds, db = qp.qcross_entropy_backward(xd, td, lse, gd, *none, 4, 32)
    assert not dx.any() and ds.shape == (0, 2)
    flat = tuple(p[:, :0].contiguous() for p in wd)
    loss, lse = qp.qcross_entropy(xd[:, :0].contiguous(), td, *flat, 4, 32)
    want = torch.tensor(40.0).log()
    assert torch.allclose(lse.cpu(), want) and torch.allclose(loss.cpu()[[0, 2]], want)


@pytest.mark.parametrize("bits,gs,m", [(3, 32, 21), (4, 64, 5)])
def test_against_differences(bits, gs, m):
    """<grad, direction> against central differences of the 64-bit loss. Their own error: the
    third derivative along a direction, below (the spread of the logits along it)^3 eps^2,
    and roundings of 2^-52 of the loss over eps."""
    k, v = 192, 50
    x, w, t, dloss = case(m, k, v, bits, gs, F32)
    xd, td, wd = x.to(dev()), t.to(dev()), oh.cuda(w)
    _, lse = qp.qcross_entropy(xd, td, *wd, bits, gs)
    out = qp.qcross_entropy_backward(xd, td, lse, dloss.to(dev()), *wd, bits, gs)
    torch.cuda.synchronize()
    g = oh.rng(5)
    q = oh.codes(w[0], bits)
    live = (t >= 0) & (t < v)
    at = torch.where(live, t.long(), 0)[:, None]
    base = [x.double(), w[1].double(), w[2].double()]

    def logits(xx, ss, bb):
        return xx @ (q * ss.repeat_interleave(gs, 1) + bb.repeat_interleave(gs, 1)).t()

    def total(*a):
        z = logits(*a)
        return float((torch.where(live, torch.logsumexp(z, 1) - z.gather(1, at)[:, 0], 0.0) * dloss.double()).sum())

    # lse is fp32: dz is off by up to p |g| (2^-23 |lse| + the lse's own bound) for it.
    _, (r_lse, b_lse), (z, *_) = forward64(x, w, t, bits, gs, F32)
    refs = backward64(x, w, t, lse.cpu(), dloss, bits, gs, F32)
    p = torch.exp(z - r_lse[:, None]) * (dloss.double() * live * (b_lse + 2.0 ** -22 * r_lse.abs()))[:, None]
    extra = [p @ oh.dense(w, bits, gs).abs(), *oh.group_sums(w, p.t() @ x.double().abs(), bits, gs)]
    eps = 1e-4
    for i, (_, bound) in enumerate(refs):
        direction = torch.randn(base[i].shape, generator=g).double()
        direction /= direction.norm()
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + eps * direction, base[i] - eps * direction
        fd = (total(*up) - total(*down)) / (2 * eps)
        spread = float((logits(*up) - logits(*down)).abs().max()) / eps
        got = float((out[i].cpu().double() * direction).sum())
        allowed = float(((bound + 1.01 * extra[i]) * direction.abs()).sum())
        allowed += spread ** 3 * eps ** 2 + 2.0 ** -50 * abs(total(*base)) / eps
        assert abs(got - fd) <= allowed, (i, got, fd, allowed)


def test_small_gradients_of_a_large_fp16_batch():
    """A mean over many rows in fp16: each dz is far below fp16's normal range, and the sums are
    right all the same."""
    m, k, v = 600, 64, 2000
    x, w, t, _ = case(m, k, v, 4, 32, F16, sigma=0.5)
    dloss = torch.full((m,), 2.0 ** -14)
    xd, td, wd = x.to(dev()), t.to(dev()), oh.cuda(w)
    _, lse = qp.qcross_entropy(xd, td, *wd, 4, 32)
    out = qp.qcross_entropy_backward(xd, td, lse, dloss.to(dev()), *wd, 4, 32)
    torch.cuda.synchronize()
    for got, (ref, bound) in zip(out, backward64(x, w, t, lse.cpu(), dloss, 4, 32, F16)):
        oh.check(got, ref, bound, "small")
