"""qcross_entropy and its backward pass where the vocabulary goes in several pieces (many rows, a
wide head, a very large vocabulary), and with weights of more than 2^31 bytes. The bounds are
those of the smaller sizes."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, HALF_SUBNORMAL, HALF_ULP, TAU, TORCH_DT, dev, log
from test_gpu_loss import run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,k,v,bits,gs,dt", [
    (16500, 64, 4100, 4, 32, BF16),      # gradients: pieces of 3840 tokens, the last of 260
    (16500, 64, 4100, 8, 64, F32),
    (33000, 64, 2300, 4, 64, F16),       # pieces of 2048
    (5000, 32, 12500, 4, 32, F32),       # short rows: pieces of 12288
    (5000, 32, 12500, 4, 32, BF16),
    (2, 64, 270001, 4, 32, BF16),        # few rows: one piece, in parts
    (16, 32, 4200000, 2, 32, BF16),      # and two pieces
])
def test_pieces(m, k, v, bits, gs, dt):
    run_and_check(m, k, v, bits, gs, dt, "pieces")


@pytest.mark.parametrize("m,k,v,dt", [
    (20, 1 << 18, 33068, BF16), (20, 1 << 18, 33068, F32), (130, 1 << 18, 33068, F16), (5, 1 << 18, 33068, BF16),
    (20, (1 << 18) + 32, 300, BF16), (3, (1 << 18) + 32, 300, F32)])
def test_the_widest_heads(m, k, v, dt):
    """2^18 features, 33068 tokens, 2 bits: 2.2 GB of codes, pieces of 16384 tokens; and the first
    width past the tiles'. x has a few features that are not 0, so that the 64-bit form needs
    only these: a product with 0 adds exactly nothing, and the sums' roundings are those of
    the others."""
    bits, gs = 2, 32
    log(f"widest head: m={m} k={k} dt={dt}")
    g = torch.Generator(device="cuda").manual_seed(m + dt)
    wq = torch.randint(-2 ** 31, 2 ** 31, (v, k * bits // 32), generator=g, device=dev(), dtype=torch.int32)
    s = ((torch.rand((v, k // gs), generator=g, device=dev()) + 0.5) * 0.25).to(TORCH_DT[dt])
    b = (-3 * s.float() * torch.rand((v, k // gs), generator=g, device=dev())).to(TORCH_DT[dt])
    at = torch.tensor([0, 31, 32, 65, 4096, 131071, 131072, k - 65, k - 33, k - 1], device=dev())
    xs = torch.randn((m, len(at)), generator=g, device=dev()).to(TORCH_DT[dt])
    x = torch.zeros((m, k), dtype=TORCH_DT[dt], device=dev())
    x[:, at] = xs
    t = torch.randint(0, v, (m,), generator=g, device=dev(), dtype=torch.int32)
    t[0], t[1] = v - 1, -100
    q = ((wq[:, at * bits // 32] >> (at * bits % 32).int()) & 3).double()
    sd, bd = s[:, at // gs].double(), b[:, at // gs].double()
    W, xd = q * sd + bd, xs.double()
    n = len(at)
    per = (3 * n + 64) * 2.0 ** -24 + (2.0 ** -17 if dt != F32 else 0.0)
    z, bz = xd @ W.t(), per * (xd.abs() @ (q * sd.abs() + bd.abs()).t())
    r_lse = torch.logsumexp(z, 1)
    b_lse = bz.max(1).values + 2.0 ** -16 + 2.0 ** -22 * r_lse.abs()
    live = (t >= 0) & (t < v)
    idx = torch.where(live, t.long(), 0)[:, None]
    loss, lse = qp.qcross_entropy(x, t, wq, s, b, bits, gs)
    torch.cuda.synchronize()
    oh.check(lse, r_lse.cpu(), b_lse.cpu(), "lse")
    r_loss = torch.where(live, r_lse - z.gather(1, idx)[:, 0], 0.0)
    b_loss = torch.where(live, b_lse + bz.gather(1, idx)[:, 0] + 2.0 ** -23 * (r_loss.abs() + r_lse.abs()), 0.0)
    oh.check(loss, r_loss.cpu(), b_loss.cpu(), "loss")

    dloss = torch.rand(m, generator=g, device=dev()) / m + 0.1 / m
    log("widest head, backward")
    dx, ds, db = qp.qcross_entropy_backward(x, t, lse, dloss, wq, s, b, bits, gs)
    torch.cuda.synchronize()
    up = torch.where(live, dloss.double(), 0.0)[:, None]
    off = z - lse.double()[:, None]
    p = torch.exp(off)
    dz = p.clone()
    dz.scatter_add_(1, idx, torch.full_like(p[:, :1], -1.0))
    dz = dz * up
    floor = HALF_SUBNORMAL[dt] * (float(up.abs().max()) * 2.0 ** -14 if dt == F16 else 1.0)
    e = up.abs() * p * (1.01 * bz + 2.0 ** -20 * (1 + off.abs())) + dz.abs() * 2.0 ** -22 + up.abs() * 2.0 ** -126
    e = torch.where(live[:, None], e + torch.clamp(1.01 * dz.abs() * HALF_ULP[dt], min=floor), 0.0)
    ref = (dz @ W).cpu()
    oh.check(dx[:, at], ref, (e @ W.abs() + TAU[dt] * (dz.abs() @ W.abs())).cpu() + oh.half_ulp(ref, dt), "dx")
    gam = oh.gamma(m + gs)
    cols = torch.zeros(k // gs, dtype=torch.bool, device=dev())
    cols[at // gs] = True
    for got, weigh, name in ((ds, q, "dscales"), (db, torch.ones_like(q), "dbiases")):
        def sums(rows, values):
            """[v, groups that x reaches] of rows^T values, times the codes or 1."""
            full = torch.zeros((v, k // gs), dtype=torch.float64, device=dev())
            return full.index_add_(1, at // gs, (rows.t() @ values) * weigh)[:, cols].cpu()
        ref = sums(dz, xd)
        oh.check(got[:, cols], ref, 1.01 * sums(e, xd.abs()) + gam * sums(dz.abs(), xd.abs()) + oh.half_ulp(ref, dt), name)
        got[:, cols] = 0
        assert not got.any(), name


def test_the_most_rows():
    """2^20 rows and more tokens than one launch of tiles takes. The rows are 64 patterns, so the
    64-bit form has 64 rows of logits."""
    if torch.cuda.get_device_properties(0).total_memory < 60 * 2 ** 30:
        pytest.skip("needs 60 GiB of GPU memory")
    m, k, v, bits, gs = 1 << 20, 64, (1 << 19) + 5, 2, 64
    log(f"most rows: {m}")
    g = oh.rng(9)
    pattern = oh.normal((64, k), 2.0, BF16, g)
    w = oh.weight(v, k, bits, gs, BF16, g)
    W = oh.dense(w, bits, gs).to(dev())
    mags = (oh.codes(w[0], bits) * oh.spread(w[1], gs).abs() + oh.spread(w[2], gs).abs()).to(dev())
    pd = pattern.to(dev()).double()
    which = torch.arange(m, device=dev()) * 37 % 64
    t = (torch.arange(m, device=dev()) * 7919 % v).to(torch.int32)
    loss, lse = qp.qcross_entropy(pattern.to(dev())[which], t, *oh.cuda(w), bits, gs)
    torch.cuda.synchronize()
    per = (k + 2 + 64) * 2.0 ** -24 + 2.0 ** -17
    r_lse = torch.logsumexp(pd @ W.t(), 1)
    b_lse = per * (pd.abs() @ mags.t()).max(1).values + 2.0 ** -16 + 2.0 ** -22 * r_lse.abs()
    at = t.long()
    r_loss = r_lse[which] - (pd[which] * W[at]).sum(1)
    b_loss = b_lse[which] + per * (pd[which].abs() * mags[at]).sum(1) + 2.0 ** -23 * (r_loss.abs() + r_lse[which].abs())
    oh.check(lse, r_lse[which].cpu(), b_lse[which].cpu(), "lse")
    oh.check(loss, r_loss.cpu(), b_loss.cpu(), "loss")
