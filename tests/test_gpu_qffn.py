"""GPU parity of qffn and qffn_backward with their 64-bit forms, and with differences.

Bounds, propagated through the block (ophelpers; TAU and half an ulp as in qhelpers):
  g, u:  B_g = TAU * |x||Wg| (+ half an ulp where stored)
  h:     B_h = 1.13 |u| B_g + |act(g)| B_u + B_g B_u + half_ulp(h); both
         activations have |act'| <= 1.13. Where the products are separate
         launches g and u are rounded first: B_g and B_u always include half an ulp.
  y:     TAU * |h||Wd| + B_h |Wd| + half_ulp(y), the first over |h| + B_h
Backward, from the given g and u:
  dh:    B = TAU * |dy||Wd| (not stored)
  dg:    |u act'| B + 2^-20 |dh u| (terms of act') + half_ulp; du: |act| B + 2^-20 |dh act| + half_ulp
  dx:    TAU * (|dg||Wg| + |du||Wu|) + B_dg |Wg| + B_du |Wu| + half_ulp(dx)
  dW:    gamma(m + gs) * |dz|^T |x| + B_dz^T |x|, summed like the gradient, + half_ulp
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, TAU, dev, log

pytestmark = pytest.mark.gpu


def case(m, d, f, bits, gs, dt):
    g = oh.rng(oh.seed_of(m, d, f, bits, gs, dt))
    c = dict(m=m, d=d, f=f, bits=bits, gs=gs, dt=dt)
    c["x"], c["dy"] = oh.normal((m, d), 1.0, dt, g), oh.normal((m, d), 0.5, dt, g)
    c["gate"], c["up"] = (oh.weight(f, d, bits, gs, dt, g) for _ in range(2))
    c["down"] = oh.weight(d, f, bits, gs, dt, g)
    return c


def forward_ref(c, act):
    dt, bits, gs = c["dt"], c["bits"], c["gs"]
    Wg, Wu, Wd = (oh.dense(c[n], bits, gs) for n in ("gate", "up", "down"))
    x = c["x"].double()
    g, u = x @ Wg.t(), x @ Wu.t()
    bg = TAU[dt] * (x.abs() @ Wg.abs().t()) + oh.half_ulp(g, dt)
    bu = TAU[dt] * (x.abs() @ Wu.abs().t()) + oh.half_ulp(u, dt)
    a = oh.act(g, act)[0]
    h = a * u
    bh = 1.13 * u.abs() * bg + a.abs() * bu + 1.13 * bg * bu + oh.half_ulp(h, dt)
    y = h @ Wd.t()
    by = TAU[dt] * ((h.abs() + bh) @ Wd.abs().t()) + bh @ Wd.abs().t() + oh.half_ulp(y, dt)
    return (y, by), (g, bg), (u, bu)


def run(c, act, saved=None):
    return qp.qffn(c["x"].to(dev()), *(oh.cuda(c[n]) for n in ("gate", "up", "down")), c["bits"],
                   c["gs"], act=act, saved=saved)


def check_forward(c, act, what):
    log(f"qffn {what}: m={c['m']} d={c['d']} f={c['f']} bits={c['bits']} gs={c['gs']} dt={c['dt']} {act}")
    (y, by), (g, bg), (u, bu) = forward_ref(c, act)
    plain = run(c, act)
    saved = torch.empty((2, c["m"], c["f"]), dtype=c["x"].dtype, device=dev())
    kept = run(c, act, saved)
    torch.cuda.synchronize()
    oh.check(plain, y, by, f"{what} y")
    oh.check(kept, y, by, f"{what} y, kept")
    oh.check(saved[0], g, bg, f"{what} g")
    oh.check(saved[1], u, bu, f"{what} u")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 17, 40, 300])
def test_forward_rows(m, dt, act):
    check_forward(case(m, 256, 448, 4, 64, dt), act, "rows")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (6, 32), (8, 32), (4, 128), (3, 64), (6, 128),
                                     (2, 64), (8, 64)])
@pytest.mark.parametrize("m", [1, 7, 33])
def test_forward_widths(m, bits, gs, dt):
    check_forward(case(m, 384, 256, bits, gs, dt), "silu", "widths")


@pytest.mark.parametrize("m,d,f", [(1, 32, 32), (1, 2080, 96), (2, 4128, 64), (1, 5632, 320), (6, 96, 1056),
                                   (18, 96, 160), (33, 32, 544), (257, 160, 96), (9, 2048, 288),
                                   (1, 8256, 64), (2, 32, 4128), (1, 17408, 32)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_forward_odd_shapes(m, d, f, dt):
    check_forward(case(m, d, f, 4, 32, dt), "silu", "odd")


@pytest.mark.parametrize("bits,gs,dt", [(2, 32, BF16), (3, 64, F16), (4, 128, BF16), (6, 32, F16), (8, 64, BF16)])
@pytest.mark.parametrize("m,d,f", [(17, 512, 1152), (64, 1152, 640), (65, 896, 1024), (129, 2048, 512),
                                   (257, 640, 2176)])
def test_forward_in_pieces(m, d, f, bits, gs, dt):
    """Few tiles and long contractions: the products in pieces, equal and not, with ends of 64-
    and 256-row tiles."""
    check_forward(case(m, d, f, bits, gs, dt), "gelu_tanh", "pieces")


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,d,f,gs", [(1, 256, 448, 64), (12, 256, 448, 64), (40, 256, 448, 64), (150, 1120, 352, 32),
                                      (33, 2144, 288, 32)])
def test_forward_misaligned(m, d, f, gs, dt):
    """Activations, scales and biases one element off every wider alignment."""
    c = case(m, d, f, 3, gs, dt)
    log(f"qffn misaligned: m={m} d={d} f={f} gs={gs} dt={dt}")

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:] = t.reshape(-1).to(dev())
        return flat[1:].view(t.shape)

    (y, by), (g, bg), (u, bu) = forward_ref(c, "silu")
    ws = [(c[n][0].to(dev()), off(c[n][1]), off(c[n][2])) for n in ("gate", "up", "down")]
    saved = off(torch.zeros((2, m, f), dtype=c["x"].dtype))
    for kept in (None, saved):
        out = off(torch.zeros((m, d), dtype=c["x"].dtype))
        qp.qffn(off(c["x"]), *ws, 3, gs, act="silu", saved=kept, out=out)
        torch.cuda.synchronize()
        oh.check(out, y, by, "y")
    oh.check(saved[0], g, bg, "g")
    oh.check(saved[1], u, bu, "u")


def backward_ref(c, saved, act):
    dt, bits, gs = c["dt"], c["bits"], c["gs"]
    Wg, Wu, Wd = (oh.dense(c[n], bits, gs) for n in ("gate", "up", "down"))
    x, dy = c["x"].double(), c["dy"].double()
    g, u = saved[0].double(), saved[1].double()
    a, da, mag = oh.act(g, act)
    dh, bdh = dy @ Wd, TAU[dt] * (dy.abs() @ Wd.abs())
    e = 2.0 ** -20
    dg, du, h = dh * u * da, dh * a, a * u
    bdg = (u * da).abs() * bdh + e * (dh.abs() + bdh) * u.abs() * mag
    bdu = a.abs() * bdh + e * (dh.abs() + bdh) * a.abs()
    bdg = bdg + oh.half_ulp(dg.abs() + bdg, dt)
    bdu = bdu + oh.half_ulp(du.abs() + bdu, dt)
    bh = e * h.abs() + oh.half_ulp(h, dt)
    dx = dg @ Wg + du @ Wu
    bdx = (TAU[dt] * ((dg.abs() + bdg) @ Wg.abs() + (du.abs() + bdu) @ Wu.abs()) + bdg @ Wg.abs()
           + bdu @ Wu.abs() + oh.half_ulp(dx, dt))
    refs = [(dx, bdx)]
    gm = oh.gamma(c["m"] + gs)
    for name, dz, bz, z, bzz in (("gate", dg, bdg, x, 0 * x), ("up", du, bdu, x, 0 * x),
                                 ("down", dy, 0 * dy, h, bh)):
        grads = oh.group_sums(c[name], dz.t() @ z, bits, gs)
        err = oh.group_sums(c[name], gm * (dz.abs() + bz).t() @ (z.abs() + bzz) + bz.t() @ (z.abs() + bzz)
                            + dz.abs().t() @ bzz, bits, gs)
        refs += [(r, b + oh.half_ulp(r, dt)) for r, b in zip(grads, err)]
    return refs


def saved_of(c):
    """What the forward pass would have kept (rounded from 64 bits)."""
    x = c["x"].double()
    return torch.stack([x @ oh.dense(c[n], c["bits"], c["gs"]).t() for n in ("gate", "up")]).to(c["x"].dtype)


def run_backward(c, saved, act, **kw):
    return qp.qffn_backward(c["x"].to(dev()), c["dy"].to(dev()), saved.to(dev()),
                            *(oh.cuda(c[n]) for n in ("gate", "up", "down")), c["bits"], c["gs"], act=act, **kw)


def check_backward(c, act, what):
    log(f"qffn_backward {what}: m={c['m']} d={c['d']} f={c['f']} bits={c['bits']} gs={c['gs']} dt={c['dt']} {act}")
    saved = saved_of(c)
    dx, *pairs = run_backward(c, saved, act)
    torch.cuda.synchronize()
    outs = [dx] + [t for p in pairs for t in p]
    names = ["dx"] + [f"{w} {p}" for w in ("gate", "up", "down") for p in ("scales", "biases")]
    for y, (ref, bound), name in zip(outs, backward_ref(c, saved, act), names):
        oh.check(y, ref, bound, f"{what} {name}")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m", [1, 5, 33, 130, 300])
def test_backward_rows(m, dt, act):
    check_backward(case(m, 256, 448, 4, 64, dt), act, "rows")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (6, 32), (8, 32), (4, 128), (8, 128)])
def test_backward_widths(bits, gs, dt):
    check_backward(case(40, 384, 256, bits, gs, dt), "gelu_tanh", "widths")


@pytest.mark.parametrize("m,d,f", [(1, 32, 32), (18, 96, 160), (33, 32, 544), (257, 160, 96), (3, 1056, 64),
                                   (600, 64, 32)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_backward_odd_shapes(m, d, f, dt):
    check_backward(case(m, d, f, 4, 32, dt), "silu", "odd")


@pytest.mark.parametrize("m,d,f,bits,gs,dt,act", [(70, 2080, 4640, 4, 32, BF16, "silu"),
                                                  (300, 1024, 1600, 6, 64, F16, "gelu_tanh"),
                                                  (520, 1536, 768, 8, 128, BF16, "gelu_tanh")])
def test_many_tiles(m, d, f, bits, gs, dt, act):
    """Blocks large enough for the persistent tiles, several a compute unit."""
    c = case(m, d, f, bits, gs, dt)
    check_backward(c, act, "many tiles")
    check_forward(c, act, "many tiles")


def test_backward_extreme_preactivations():
    """Gates far out on both sides: the derivative's terms vanish or stay, nothing is NaN."""
    c = case(4, 64, 64, 4, 32, F32)
    saved = saved_of(c)
    far = torch.tensor([-3e38, -1e20, -200.0, -88.0, -20.0, 0.0, 20.0, 88.0, 1e20, 3e38])
    for act in ("silu", "gelu_tanh"):
        s = saved.clone()
        s[0, :, :10] = far
        s[1] = 1.0
        dx, *pairs = run_backward(c, s, act)
        (dh,) = (c["dy"].double() @ oh.dense(c["down"], 4, 32),)
        # du = dh act(g) overflows only where act(g) dh does.
        assert not dx.isnan().any() or (dh * 3e38).abs().max() > 3.4e38
        ref = oh.act(s[0].double(), act)[1]
        assert torch.isfinite(ref).all()
        s[0, :, 0], s[0, :, 8:10] = -50.0, 50.0
        dx, *pairs = run_backward(c, s, act)
        assert torch.isfinite(dx).all() and all(torch.isfinite(t).all() for p in pairs for t in p)


def test_backward_deterministic_and_parts():
    c = case(70, 256, 320, 4, 64, BF16)
    saved = saved_of(c)
    a, b = run_backward(c, saved, "silu"), run_backward(c, saved, "silu")
    frozen = run_backward(c, saved, "silu", weight_grads=False)
    params = run_backward(c, saved, "silu", input_grad=False)
    torch.cuda.synchronize()
    assert oh.same_bits(a[0], b[0]) and oh.same_bits(a[0], frozen[0]) and frozen[1:] == (None, None, None)
    assert params[0] is None
    for i in (1, 2, 3):
        for j in (0, 1):
            assert oh.same_bits(a[i][j], b[i][j]) and oh.same_bits(a[i][j], params[i][j])


def test_empty():
    c = case(3, 64, 96, 4, 32, BF16)
    w = [oh.cuda(c[n]) for n in ("gate", "up", "down")]
    x = c["x"].to(dev())
    assert qp.qffn(x[:0], *w, 4, 32).shape == (0, 64)
    saved = torch.empty((2, 0, 96), dtype=torch.bfloat16, device=dev())
    dx, *pairs = qp.qffn_backward(x[:0], x[:0], saved, *w, 4, 32)
    assert dx.shape == (0, 64) and not any(t.any() for p in pairs for t in p)
    none = [tuple(t[:0] for t in w[0]), tuple(t[:0] for t in w[1]), tuple(t[:, :0].contiguous() for t in w[2])]
    assert not qp.qffn(x, *none, 4, 32).any()
    dx, *_ = qp.qffn_backward(x, x, saved.new_empty((2, 3, 0)), *none, 4, 32)
    assert not dx.any()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_against_differences(act):
    """<grad, direction> against central differences of the 64-bit block. With
    eps = 1e-4 the third-order term is below 1e-7 of the sum of magnitudes."""
    c = case(9, 96, 160, 4, 32, F32)
    bits, gs = 4, 32
    x = c["x"].double()
    q = {n: oh.codes(c[n][0], bits) for n in ("gate", "up", "down")}
    p = {(n, i): c[n][1 + i].double() for n in q for i in (0, 1)}

    def loss(xx, pp):
        W = {n: q[n] * pp[n, 0].repeat_interleave(gs, 1) + pp[n, 1].repeat_interleave(gs, 1) for n in q}
        g, u = xx @ W["gate"].t(), xx @ W["up"].t()
        return float((c["dy"].double() * ((oh.act(g, act)[0] * u) @ W["down"].t())).sum())

    saved = torch.empty((2, 9, 160), dtype=torch.float32, device=dev())
    run(c, act, saved)
    dx, *pairs = run_backward(c, saved, act)
    refs = backward_ref(c, saved.cpu(), act)
    grads = {"x": (dx, refs[0][1])}
    for k, n in enumerate(("gate", "up", "down")):
        for i in (0, 1):
            grads[n, i] = (pairs[k][i], refs[1 + 2 * k + i][1])
    gen, eps = oh.rng(11), 1e-4
    (y, by), (g, bg), (u, bu) = forward_ref(c, act)
    for name, (grad, bound) in grads.items():
        base = x if name == "x" else p[name]
        scale = 1.0 if name == "x" else 0.05
        dr = torch.randn(base.shape, generator=gen).double() * scale
        def at(t):
            return loss(x + t * dr, p) if name == "x" else loss(x, {**p, name: base + t * dr})
        fd = (at(eps) - at(-eps)) / (2 * eps)
        got = grad.cpu().double()
        tol = float((bound * dr.abs()).sum()) + 1e-6 * float((got.abs() * dr.abs()).sum())
        # The saved products' own rounding moves the point the gradient is taken at.
        tol += 1e-5 * float((got.abs() * dr.abs()).sum())
        assert abs(float((got * dr).sum()) - fd) <= tol, (name, float((got * dr).sum()), fd, tol)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("bits", [2, 3, 6, 8])
@pytest.mark.parametrize("m,d,f", [(17, 96, 160), (40, 1120, 352), (130, 352, 1120), (300, 160, 2080), (64, 2080, 96)])
def test_forward_filled_up_contractions(m, d, f, bits, dt):
    """Both contractions of 64 n + 32, at the widths whose rows of codes end inside a 16-byte
    piece (2 and 6) and at those that do not. Every code occurs, the last row's last ones too."""
    c = case(m, d, f, bits, 32, dt)
    for n in ("gate", "up", "down"):
        assert (oh.codes(c[n][0], bits)[-1, -32:] != 0).any()
    check_forward(c, "silu", "filled up")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("m,d,f", [(4, 64, 64), (40, 96, 160), (300, 128, 192)])
def test_backward_far_preactivations_against_the_formula(m, d, f, dt, act):
    """Gates at the ends of the type's range, one column each (so a row each of the gate's and
    up's gradients): every gradient against the 64-bit form. dy is small enough, and u there
    one half, so that nothing leaves the range."""
    c = case(m, d, f, 4, 32, dt)
    top, small = (60000.0, 1e-3) if dt == F16 else (3e38, 1e-30)
    c["dy"] = (c["dy"].double() * small).to(c["dy"].dtype)
    far = [-top, -top / 4, -1e4, -200.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 200.0, 1e4, top / 4, top]
    saved = saved_of(c)
    saved[0, :, :len(far)] = torch.tensor(far, dtype=torch.float64).to(saved.dtype)
    saved[1, :, :len(far)] = 0.5
    log(f"qffn_backward far pre-activations: m={m} d={d} f={f} dt={dt} {act}")
    dx, *pairs = run_backward(c, saved, act)
    torch.cuda.synchronize()
    outs = [dx] + [t for p in pairs for t in p]
    names = ["dx"] + [f"{w} {p}" for w in ("gate", "up", "down") for p in ("scales", "biases")]
    for y, (ref, bound), name in zip(outs, backward_ref(c, saved, act), names):
        assert torch.isfinite(ref).all() and torch.isfinite(bound).all()
        oh.check(y, ref, bound, f"far {name}")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("m,d,f", [(40, 256, 448), (300, 1024, 640), (5, 4096, 96)])
def test_backward_alignment_changes_nothing(m, d, f, dt):
    c = case(m, d, f, 4, 32, dt)
    saved = saved_of(c)
    want = run_backward(c, saved, "silu")

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:] = t.reshape(-1).to(dev())
        return flat[1:].view(t.shape)

    ws = [tuple(off(t) for t in c[n]) for n in ("gate", "up", "down")]
    log(f"qffn_backward at other addresses: m={m} d={d} f={f} dt={dt}")
    got = qp.qffn_backward(off(c["x"]), off(c["dy"]), off(saved), *ws, c["bits"], c["gs"], act="silu")
    torch.cuda.synchronize()
    assert oh.same_bits(got[0], want[0])
    assert all(oh.same_bits(a, b) for p, q in zip(got[1:], want[1:]) for a, b in zip(p, q))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_backward_single_pairs_through_the_c_abi(dt, act):
    """Each weight's gradients asked for alone, with the pointers that they do not need null or
    absent: the same bits as with everything, and the down pair's without the weights read."""
    c = case(50, 256, 320, 4, 64, dt)
    saved = saved_of(c).to(dev())
    want = run_backward(c, saved.cpu(), act)
    x, dy = c["x"].to(dev()), c["dy"].to(dev())
    ws = [t for n in ("gate", "up", "down") for t in oh.cuda(c[n])]
    work = torch.empty(qp.qffn_backward_workspace_bytes(50, 256, 320, 4, 64, x.dtype), dtype=torch.uint8, device=dev())
    log(f"qffn_backward, one pair at a time: dt={dt} {act}")
    for i in range(3):
        pair = [torch.full_like(t, 7.0) for t in want[1 + i]]
        grads = [None] * 6
        grads[2 * i], grads[2 * i + 1] = (t.data_ptr() for t in pair)
        # dh overwrites dg and du: with the down pair alone they stay as they were.
        work.fill_(1)
        qp.check(qp.lib().qffn_backward(
            x.data_ptr() if i < 2 else None, dy.data_ptr(), saved.data_ptr(), dt, 50, 256, 320,
            *[t.data_ptr() for t in ws], dt, 4, 64, qp.ACTS[act], None, *grads, work.data_ptr(), work.numel(), None))
        torch.cuda.synchronize()
        assert all(oh.same_bits(a, b) for a, b in zip(pair, want[1 + i])), i
        mf = 50 * 320 * x.element_size()          # a multiple of 16: dg, then du
        if i == 2:
            assert (work[:2 * mf] == 1).all()
