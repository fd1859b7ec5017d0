"""GPU parity of qblock_norm and its backward pass with their 64-bit forms, and with
differences.

Everything is fp32 from the loads on, so a value made of terms of magnitude T, with sums
over a row of d (or m rows), is within C 2^-24 T of its 64-bit form, C = d + 64 (m + 64)
roundings in a row at most, and half an ulp of its own rounding.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev, log

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]   # the block's, the stream's


class Case:
    def __init__(self, m, d, dt, sdt, post, gates, pre, offset=0.0, y=True, seed=0):
        g = oh.rng(oh.seed_of(m, d, dt, sdt, post, gates, pre, offset, y, seed))
        self.m, self.d, self.dt, self.sdt, self.offset, self.factor = m, d, dt, sdt, offset, 0.75
        self.x = oh.normal((m, d), 3.0, sdt, g)
        if d > 9:
            self.x[:, 7] *= 20
        self.y = oh.normal((m, d), 2.0, dt, g) if y else None

        def weight(n):
            return (torch.randn(n, generator=g) * 0.3 + 1 - offset).to(self.x.dtype if dt == sdt else oh.TORCH_DT[dt])

        self.post = weight((d,)) if post else None
        self.weight = weight((d,)) if pre else None
        self.gate = oh.normal((gates, d), 0.7, dt, g) if gates else None
        self.ds = oh.normal((m, d), 0.3, sdt, g)
        self.da = oh.normal((m, d), 0.3, dt, g) if pre else None

    def parts(self, move=lambda t: t.to(dev())):
        names = ("y", "weight", "gate")
        out = {n: None if getattr(self, n) is None else move(getattr(self, n)) for n in names}
        out["post_weight"] = None if self.post is None else move(self.post)
        return {**out, "scale": self.factor, "offset": self.offset, "eps": EPS}

    def forward64(self):
        """(ref, bound) of s and a, None for what there is not."""
        x, C = self.x.double(), (self.d + 64) * 2.0 ** -24
        s, T = x, x.abs()
        if self.y is not None:
            t = self.y.double()
            if self.post is not None:
                t = t / rms(t) * (self.post.double() + self.offset)
            if self.gate is not None:
                t = t * self.gate.double().repeat_interleave(self.m // self.gate.shape[0], 0)
            s, T = x + self.factor * t, T + (self.factor * t).abs()
        out = [(s, C * T + oh.half_ulp(s, self.sdt)) if self.y is not None else None]
        if self.weight is None:
            return out + [None]
        k = (self.weight.double() + self.offset) / rms(s)
        a = s * k
        # s is off by C T: in its own place, and through the mean square.
        through = (s.abs() * T).mean(1, keepdim=True) / rms(s) ** 2
        return out + [(a, 2 * C * (T * k.abs() + a.abs() * (1 + through)) + oh.half_ulp(a, self.dt))]

    def backward64(self, s):
        """(ref, bound) of dx, dy, dweight, dpost, dgate at the stream s that was written."""
        C, R = 4 * (self.d + 64) * 2.0 ** -24, (self.m + 64) * 2.0 ** -24
        G = self.ds.double()
        T = G.abs()
        out = [None] * 5
        if self.weight is not None:
            v, da, w = s.double(), self.da.double(), self.weight.double() + self.offset
            r = 1 / rms(v)
            u = da * w
            G = G + r * u - v * r ** 3 * (u * v).mean(1, keepdim=True)
            T = T + r * u.abs() + v.abs() * r ** 3 * (u * v).abs().mean(1, keepdim=True)
            dw = da * v * r
            out[2] = self.sums(dw.sum(0), dw.abs().sum(0), C + R)
        out[0] = (G, C * T + oh.half_ulp(G, self.sdt))
        if self.y is None:
            return out
        y = self.y.double()
        r = 1 / rms(y)
        n, wp = (y * r, self.post.double() + self.offset) if self.post is not None else (y, 1.0)
        gate = 1.0
        if self.gate is not None:
            rows, each = self.gate.shape[0], self.m // self.gate.shape[0]
            gate = self.gate.double().repeat_interleave(each, 0)
            dg = self.factor * n * wp * G
            mags = (self.factor * n * wp).abs() * T
            out[4] = self.sums(dg.reshape(rows, each, -1).sum(1), mags.reshape(rows, each, -1).sum(1), 2 * C + R)
        q, qT = self.factor * gate * G, (self.factor * gate * T if self.gate is None else (self.factor * gate).abs() * T)
        if self.post is None:
            out[1] = (q, 2 * C * qT + oh.half_ulp(q, self.dt))
            return out
        out[3] = self.sums((q * n).sum(0), (qT * n.abs()).sum(0), 2 * C + R)
        u, uT = q * wp, qT * wp.abs()
        dy = r * u - y * r ** 3 * (u * y).mean(1, keepdim=True)
        dyT = r * uT + y.abs() * r ** 3 * (uT * y.abs()).mean(1, keepdim=True)
        out[1] = (dy, 3 * C * dyT + oh.half_ulp(dy, self.dt))
        return out

    def sums(self, ref, mags, c):
        return ref, c * mags + oh.half_ulp(ref, self.dt)


def rms(v):
    return torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def check(got, ref, bound, dt, what):
    """oh.check; and in fp16, whose largest value is 65504 and whose step there is 32, what is
    65520 or more away from zero rounds to an infinity of its sign (the row of zeros below has
    gradients of 1 / sqrt(eps) times their like)."""
    over = (ref.abs() - bound >= 65520.0) if dt == F16 else torch.zeros_like(ref, dtype=torch.bool)
    assert torch.equal(got.cpu().double()[over], torch.inf * ref[over].sign()), what
    oh.check(torch.where(over.to(dev()), 0, got), torch.where(over, 0.0, ref), bound, what)


def run_and_check(c, what, move=lambda t: t.to(dev())):
    log(f"qblock_norm {what}: m={c.m} d={c.d} dt={c.dt} sdt={c.sdt} post={c.post is not None} "
        f"gate={None if c.gate is None else c.gate.shape[0]} pre={c.weight is not None} y={c.y is not None}")
    x = move(c.x)
    s, a = qp.qblock_norm(x, **c.parts(move))
    torch.cuda.synchronize()
    for got, want, name in zip((s, a), c.forward64(), ("s", "a")):
        if want is not None:
            check(got, *want, c.sdt if name == "s" else c.dt, f"{what} {name}")
    assert (s is x) == (c.y is None) and (a is None) == (c.weight is None)
    out = qp.qblock_norm_backward(s, None if c.da is None else move(c.da), move(c.ds), **c.parts(move))
    torch.cuda.synchronize()
    for got, want, name in zip(out, c.backward64(s.cpu()), ("dx", "dy", "dweight", "dpost", "dgate")):
        assert (got is None) == (want is None), name
        if want is not None:
            check(got, *want, c.sdt if name == "dx" else c.dt, f"{what} {name}")


@pytest.mark.parametrize("dt,sdt", TYPES)
@pytest.mark.parametrize("d", [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 1024, 1025, 2047, 2048, 2049, 2881, 4096,
                               4100, 5120, 8191, 8192, 8193, 16384])
def test_widths(d, dt, sdt):
    run_and_check(Case(3, d, dt, sdt, True, 1, True), "widths")


@pytest.mark.parametrize("dt,sdt", TYPES)
@pytest.mark.parametrize("post,gates,pre,y", [
    (True, 0, True, True), (False, 0, True, True), (True, 0, False, True), (False, 0, False, True), (False, 0, True, False),
    (False, 1, True, True), (True, 1, False, True), (False, 4, True, True), (True, 12, True, True), (True, 6, False, True)])
def test_every_combination_of_parts(post, gates, pre, y, dt, sdt):
    for offset in (0.0, 1.0):
        run_and_check(Case(12, 200, dt, sdt, post, gates, pre, offset, y), "parts")


@pytest.mark.parametrize("m,gates", [(1, 1), (2, 2), (5, 0), (64, 1), (511, 1), (513, 1), (600, 600), (1030, 515), (1200, 4),
                                     (2048, 256), (1026, 513), (1500, 3)])
def test_rows_and_gates(m, gates):
    """Few rows and many, fewer gate rows than blocks and more."""
    run_and_check(Case(m, 136, BF16, BF16, True, gates, True), "rows")
    run_and_check(Case(m, 33, F32, F32, True, gates, True), "rows")


@pytest.mark.parametrize("m,d,gates", [(700, 1027, 1), (520, 4096, 4), (520, 4096, 520), (24, 8200, 2), (24, 8200, 24),
                                       (600, 8300, 600)])
def test_larger(m, d, gates):
    run_and_check(Case(m, d, BF16, F32, True, gates, True), "larger")


def shifted(t):
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
    flat[1:] = t.flatten().to(dev())
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dt,sdt", TYPES)
@pytest.mark.parametrize("d", [96, 2050])
def test_misaligned_bases(d, dt, sdt):
    run_and_check(Case(5, d, dt, sdt, True, 5, True), "misaligned", move=shifted)


@pytest.mark.parametrize("dt,sdt", TYPES)
def test_in_place(dt, sdt):
    c = Case(9, 520, dt, sdt, True, 1, True)
    want = qp.qblock_norm(c.x.to(dev()), **c.parts())
    x, parts = c.x.to(dev()), c.parts()
    got = qp.qblock_norm(x, **parts, stream=x, out=parts["y"])
    torch.cuda.synchronize()
    assert got[0] is x and got[1] is parts["y"] and oh.same_bits(got[0], want[0]) and oh.same_bits(got[1], want[1])


def test_without_ds_and_twice():
    c = Case(40, 300, BF16, F32, True, 4, True)
    s, _ = qp.qblock_norm(c.x.to(dev()), **c.parts())
    zeros = torch.zeros_like(s)
    runs = [qp.qblock_norm_backward(s, c.da.to(dev()), ds, **c.parts()) for ds in (None, zeros, zeros)]
    torch.cuda.synchronize()
    assert all(oh.same_bits(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_empty(dt):
    c = Case(4, 64, dt, dt, True, 1, True)
    parts = c.parts()
    parts["y"] = parts["y"][:0]
    s, a = qp.qblock_norm(c.x[:0].to(dev()), **parts)
    assert s.shape == a.shape == (0, 64)
    dx, dy, dw, dp, dg = qp.qblock_norm_backward(s, a, s, **parts)
    torch.cuda.synchronize()
    assert dx.shape == dy.shape == (0, 64) and not dw.any() and not dp.any() and not dg.any()


@pytest.mark.parametrize("dt,sdt", TYPES)
def test_zero_rows_and_nan(dt, sdt):
    """A row of zeros norms to zeros; a NaN stays in its row, and in the sums over rows."""
    c = Case(6, 700, dt, sdt, True, 6, True)
    c.y[2] = 0
    c.x[2] = 0
    run_and_check(c, "zero row")
    want = qp.qblock_norm(c.x.to(dev()), **c.parts())
    c.y[4, 699] = float("nan")
    s, a = qp.qblock_norm(c.x.to(dev()), **c.parts())
    dx, dy, dw, dp, dg = qp.qblock_norm_backward(s, c.da.to(dev()), c.ds.to(dev()), **c.parts())
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 5]
    assert oh.same_bits(s[keep], want[0][keep]) and oh.same_bits(a[keep], want[1][keep])
    assert s[4].isnan().all() and a[4].isnan().all() and dx[4].isnan().all() and dy[4].isnan().all()
    assert not (dx[keep].isnan().any() or dy[keep].isnan().any() or dg[keep].isnan().any())
    assert dw.isnan().all() and dp.isnan().all() and dg[4].isnan().all()


@pytest.mark.parametrize("gates", [0, 1, 3, 9])
def test_against_differences(gates):
    """<grad, direction> against central differences of the 64-bit forward pass. Their own
    error is below eps^2 times the third derivative (of order 1 for unit directions and
    streams of this size, taken as 1e3) and 2^-50 of the sum over eps."""
    c = Case(9, 50, F32, F32, True, gates, True)
    s, _ = qp.qblock_norm(c.x.to(dev()), **c.parts())
    grads = qp.qblock_norm_backward(s, c.da.to(dev()), c.ds.to(dev()), **c.parts())
    torch.cuda.synchronize()
    names = ["x", "y", "weight", "post"] + (["gate"] if gates else [])
    keep = {n: getattr(c, n) for n in names}
    bounds = [b for _, b in (p for p in c.backward64(c.forward64()[0][0]) if p is not None)]

    def total():
        (rs, _), (ra, _) = c.forward64()
        return float((rs * c.ds.double()).sum() + (ra * c.da.double()).sum())

    g, eps = oh.rng(3), 1e-5
    for i, n in enumerate(names):
        direction = torch.randn(keep[n].shape, generator=g).double()
        direction /= direction.norm()
        values = []
        for sign in (1, -1):
            setattr(c, n, keep[n].double() + sign * eps * direction)
            values.append(total())
        setattr(c, n, keep[n])
        fd = (values[0] - values[1]) / (2 * eps)
        got = float((grads[i].cpu().double() * direction).sum())
        # s was written in fp32: its half ulp goes through the same bounds once more.
        allowed = 2 * float((bounds[i] * direction.abs()).sum()) + 1e3 * eps ** 2 + 2.0 ** -50 * 500 / eps
        assert abs(got - fd) <= allowed, (n, got, fd, allowed)
