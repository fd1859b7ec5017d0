"""qffn's hidden values come from fp32 projections, whatever kernel takes the shape.

Exact cases: one weight row of gate and up gives projections that fp32 holds and the
operator's 16-bit type does not, and every sum on the way is exact, so y is one number.
With g and u rounded to the type before the activation it would be another (and in fp16
a projection beyond 65504 an infinity). Both activations are the identity (to 2^-24) on
the gates used, or zero. And y has the same bits with and without the projections kept.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, TORCH_DT, dev, log

pytestmark = pytest.mark.gpu

# m, d, f, gs: the row kernels (1 and 2 rows), one row of more than 8192, the skinny kernel,
# pieces, tiles, a contraction of 32, and filled-up contractions.
SHAPES = [(1, 256, 448, 64), (1, 4096, 64, 64), (1, 8256, 64, 32), (1, 17408, 64, 64), (2, 256, 448, 64),
          (2, 4160, 64, 32), (3, 256, 448, 64), (7, 8320, 128, 128), (16, 384, 256, 128), (17, 256, 448, 64),
          (40, 1120, 352, 32), (33, 32, 544, 32), (5, 32, 96, 32), (300, 256, 448, 64), (600, 512, 8192, 64)]


def packed(n, k, gs, dt, entries):
    """8-bit weights [n, k] of scale 1 and bias 0: entries (row, column, code), zeros elsewhere."""
    q = torch.zeros((n, k), dtype=torch.uint8)
    for r, c, code in entries:
        q[r, c] = code
    one = torch.ones((n, k // gs), dtype=TORCH_DT[dt])
    return q.view(torch.int32).reshape(n, k // 4), one, torch.zeros_like(one)


def exact_case(m, d, f, gs, dt, g, u):
    """x, weights: projection f - 1 is g times, u times x's last two columns' values."""
    x = torch.zeros((m, d), dtype=TORCH_DT[dt])
    x[:, d - 1], x[:, d - 2], x[:, 0], x[:, 1] = g[1], 1.0, u[1], 1.0
    gate = packed(f, d, gs, dt, [(f - 1, d - 1, g[0]), (f - 1, d - 2, g[2])])
    up = packed(f, d, gs, dt, [(f - 1, 0, u[0]), (f - 1, 1, u[2])])
    down = packed(d, f, gs, dt, [(5, f - 1, 1)])
    return x, gate, up, down


def shifted(t):
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
    flat[1:] = t.reshape(-1).to(dev())
    return flat[1:].view(t.shape)


def run_exact(m, d, f, gs, dt, g, u, act, off):
    """y's column 5 of every row, without and with the projections kept, and those."""
    x, *ws = exact_case(m, d, f, gs, dt, g, u)
    move = shifted if off else (lambda t: t.to(dev()))
    ws = [(w[0].to(dev()), move(w[1]), move(w[2])) for w in ws]
    saved = move(torch.full((2, m, f), 9.0, dtype=x.dtype))
    y = qp.qffn(move(x), *ws, 8, gs, act=act)
    kept = qp.qffn(move(x), *ws, 8, gs, act=act, saved=saved)
    torch.cuda.synchronize()
    assert oh.same_bits(y, kept), "with and without the projections kept"
    rest = y.clone()
    rest[:, 5] = 0
    assert not rest.any()
    return y[:, 5].cpu(), saved.cpu()


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("m,d,f,gs", SHAPES)
def test_projections_are_not_rounded(m, d, f, gs, dt, act, off):
    log(f"exact block m={m} d={d} f={f} gs={gs} dt={dt} {act} misaligned={off}")
    # bf16 (8 bits): g = 257, u = 129, h = 33153 -> 33152; from g = 256 it would be 33024.
    # fp16 (11 bits): g = 2049, u = 31, h = 63519 -> 63520; from g = 2048 it would be 63488.
    g, u, h = ((255, 1.0, 2), (127, 1.0, 2), 33152.0) if dt == BF16 else ((255, 8.0, 9), (30, 1.0, 1), 63520.0)
    y, saved = run_exact(m, d, f, gs, dt, g, u, act, off)
    assert (y == h).all(), (float(y[0]), h)
    values = [g[0] * g[1] + g[2], u[0] * u[1] + u[2]]
    want = torch.zeros((2, m, f), dtype=torch.float32)
    want[0, :, f - 1], want[1, :, f - 1] = values
    assert torch.equal(saved, want.to(saved.dtype))


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("m,d,f,gs", SHAPES)
def test_projections_beyond_half_precision(m, d, f, gs, off):
    """g = -+76800: act(g) is 0 or g, and u = 2^-4 brings h back into the type."""
    log(f"block beyond fp16 m={m} d={d} f={f} gs={gs} misaligned={off}")
    for sign in (-1.0, 1.0):
        y, saved = run_exact(m, d, f, gs, F16, (240, 320.0 * sign, 0), (1, 2.0 ** -4, 0), "silu", off)
        assert (y == (0.0 if sign < 0 else 4800.0)).all(), float(y[0])
        assert torch.isinf(saved[0, :, f - 1]).all() and (saved[1, :, f - 1] == 2.0 ** -4).all()


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("bits,gs", [(4, 64), (3, 32), (6, 64), (2, 128), (8, 32)])
@pytest.mark.parametrize("m", [1, 2, 4, 16, 23, 150])
def test_keeping_the_projections_changes_nothing(m, bits, gs, dt):
    g = oh.rng(oh.seed_of(m, bits, gs, dt, "keep"))
    d, f = 384, 640
    x = oh.normal((m, d), 1.0, dt, g).to(dev())
    ws = [oh.cuda(oh.weight(n, k, bits, gs, dt, g)) for n, k in ((f, d), (f, d), (d, f))]
    saved = torch.empty((2, m, f), dtype=x.dtype, device=dev())
    log(f"block kept or not m={m} bits={bits} gs={gs} dt={dt}")
    y, kept = qp.qffn(x, *ws, bits, gs), qp.qffn(x, *ws, bits, gs, saved=saved)
    torch.cuda.synchronize()
    assert oh.same_bits(y, kept)


def test_more_rows_than_one_pass():
    """g and u of 2 GB and more: the rows go in passes, the last one shorter, with the same
    result for every row; u is kept where it belongs."""
    m, d, f, gs = 70000, 64, 16384, 64
    x, *ws = exact_case(1, d, f, gs, BF16, (255, 1.0, 2), (127, 1.0, 2))
    ws = [oh.cuda(w) for w in ws]
    sign = torch.where(torch.arange(m, device=dev()) % 3 == 0, -1.0, 1.0).to(torch.bfloat16)
    rows = x.to(dev()).expand(m, d).clone()
    rows[:, :2] *= sign[:, None]                  # u, and so y, changes its sign
    log(f"exact block m={m} d={d} f={f} in passes")
    saved = torch.empty((2, m, f), dtype=rows.dtype, device=dev())
    for kept in (None, saved):
        y = qp.qffn(rows, *ws, 8, gs, saved=kept)
        torch.cuda.synchronize()
        assert (y[:, 5] == 33152.0 * sign).all() and not y[:, :5].any() and not y[:, 6:].any()
    # 257 and 129 in eight bits.
    assert (saved[0, :, f - 1] == 256.0).all() and (saved[1, :, f - 1] == 129.0 * sign).all()
    assert not saved[:, :, :f - 1].any()


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("bits,gs", [(4, 64), (3, 32), (8, 32)])
@pytest.mark.parametrize("m", [1, 2, 5, 16, 40, 150])
def test_alignment_changes_nothing(m, bits, gs, dt):
    g = oh.rng(oh.seed_of(m, bits, gs, dt, "address"))
    d, f = 384, 640
    x = oh.normal((m, d), 1.0, dt, g)
    ws = [oh.weight(n, k, bits, gs, dt, g) for n, k in ((f, d), (f, d), (d, f))]
    log(f"block at other addresses m={m} bits={bits} gs={gs} dt={dt}")
    y = qp.qffn(x.to(dev()), *(oh.cuda(w) for w in ws), bits, gs)
    off = qp.qffn(shifted(x), *(tuple(shifted(t) for t in w) for w in ws), bits, gs)
    torch.cuda.synchronize()
    assert oh.same_bits(y, off)
