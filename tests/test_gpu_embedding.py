"""GPU parity of qembedding and qembedding_backward with their 64-bit forms.

Bounds: lookup: w = q s + b in fp32 and one product with the factor, 4 roundings of
2^-24 of (|q s| + |b|) |factor|, and half an ulp. Gradient: the terms are exact, so
gamma(tokens of the row + gs) * the sum of magnitudes, and half an ulp.
"""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev, log

pytestmark = pytest.mark.gpu


def table(v, k, bits, gs, dt):
    return oh.weight(v, k, bits, gs, dt, oh.rng(oh.seed_of(v, k, bits, gs, dt)))


def check_lookup(ids, w, bits, gs, dt, factor, what):
    v, k = w[1].shape[0], w[1].shape[1] * gs
    out = qp.qembedding(ids.to(dev()), *oh.cuda(w), bits, gs, factor=factor)
    torch.cuda.synchronize()
    flat = ids.flatten().long()
    live = (flat >= 0) & (flat < v)
    at = flat.clamp(0, max(v - 1, 0))
    rows = tuple(t[at] for t in w)
    ref = oh.dense(rows, bits, gs) * factor * live[:, None]
    mag = (oh.codes(rows[0], bits) * oh.spread(rows[1], gs).abs() + oh.spread(rows[2], gs).abs()) * abs(factor)
    oh.check(out, ref.reshape(*ids.shape, k),
             (4 * 2.0 ** -24 * mag + oh.half_ulp(ref, dt)).reshape(*ids.shape, k), what)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (4, 64), (6, 32), (8, 128), (3, 128), (6, 64)])
def test_lookup_widths(bits, gs, dt):
    w = table(50, 384, bits, gs, dt)
    ids = torch.randint(0, 50, (3, 7), generator=oh.rng(1)).to(torch.int32)
    log(f"lookup bits={bits} gs={gs} dt={dt}")
    check_lookup(ids, w, bits, gs, dt, 1.0, "lookup")
    check_lookup(ids, w, bits, gs, dt, -11.3137085, "lookup with a factor")


@pytest.mark.parametrize("t,v,k", [(1, 1, 32), (1, 1000, 4096), (5, 3, 96), (1000, 100, 160), (300, 17, 2080)])
def test_lookup_sizes(t, v, k):
    w = table(v, k, 4, 32, BF16)
    ids = torch.randint(0, v, (t,), generator=oh.rng(t)).to(torch.int32)
    ids[-1] = v - 1
    check_lookup(ids, w, 4, 32, BF16, 1.0, "sizes")


def test_lookup_outside_ids_misaligned_out_and_empty():
    w = table(20, 64, 4, 32, F16)
    ids = torch.tensor([0, 19, 20, -1, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32)
    check_lookup(ids, w, 4, 32, F16, 2.0, "outside")
    flat = torch.full((7 * 64 + 1,), 3.0, dtype=torch.float16, device=dev())
    out = flat[1:].view(7, 64)
    ref = qp.qembedding(ids.to(dev()), *oh.cuda(w), 4, 32)
    qp.qembedding(ids.to(dev()), *oh.cuda(w), 4, 32, out=out)
    torch.cuda.synchronize()
    assert oh.same_bits(out, ref) and float(flat[0]) == 3.0
    assert qp.qembedding(ids[:0].to(dev()), *oh.cuda(w), 4, 32).shape == (0, 64)


def check_grad(ids, w, bits, gs, dt, factor, what):
    v, k = w[1].shape[0], w[1].shape[1] * gs
    t = ids.numel()
    dout = oh.normal((*ids.shape, k), 1.0, dt, oh.rng(oh.seed_of(what, t, k)))
    ds, db = qp.qembedding_backward(ids.to(dev()), dout.to(dev()), w[0].to(dev()), bits, gs, factor=factor)
    again = qp.qembedding_backward(ids.to(dev()), dout.to(dev()), w[0].to(dev()), bits, gs, factor=factor)
    torch.cuda.synchronize()
    assert oh.same_bits(ds, again[0]) and oh.same_bits(db, again[1])
    flat = ids.flatten().long()
    live = (flat >= 0) & (flat < v)
    rows = dout.reshape(t, k).double()[live]
    D = torch.zeros((v, k), dtype=torch.float64).index_add_(0, flat[live], rows)
    A = torch.zeros((v, k), dtype=torch.float64).index_add_(0, flat[live], rows.abs())
    most = int(torch.bincount(flat[live], minlength=1).max()) if live.any() else 0
    for got, ref, mag in zip((ds, db), oh.group_sums(w, D, bits, gs), oh.group_sums(w, A, bits, gs)):
        ref, mag = ref * factor, mag * abs(factor)
        bound = oh.gamma(most + gs) * mag + oh.half_ulp(ref, dt)
        bound[mag == 0] = 0.0          # rows without tokens are exactly zero
        oh.check(got, ref, bound, what)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("bits,gs", [(2, 32), (3, 32), (4, 64), (6, 32), (8, 128), (3, 128)])
def test_grad_widths(bits, gs, dt):
    w = table(40, 384, bits, gs, dt)
    ids = torch.randint(0, 30, (4, 25), generator=oh.rng(2)).to(torch.int32)
    log(f"embedding grad bits={bits} gs={gs} dt={dt}")
    check_grad(ids, w, bits, gs, dt, 1.5, "grad widths")


@pytest.mark.parametrize("t,v,k", [(1, 1, 32), (2, 9, 96), (31, 4, 160), (32, 1, 64), (33, 1, 64), (65, 2, 544),
                                   (2047, 300, 64), (2048, 300, 64), (2049, 300, 64), (4096, 7, 32),
                                   (5000, 4000, 96), (9000, 2, 64), (700, 50, 4128)])
def test_grad_sizes_and_runs(t, v, k):
    """Runs of every length around the pieces and the sorted chunks."""
    w = table(v, k, 4, 32, BF16)
    ids = torch.randint(0, v, (t,), generator=oh.rng(t)).to(torch.int32)
    log(f"embedding grad t={t} v={v} k={k}")
    check_grad(ids, w, 4, 32, BF16, 1.0, "grad sizes")


@pytest.mark.parametrize("t", [100, 3000])
def test_grad_one_hot_token_among_many(t):
    v = 500
    w = table(v, 64, 8, 32, F32)
    ids = torch.randint(0, v, (t,), generator=oh.rng(3)).to(torch.int32)
    ids[torch.rand(t, generator=oh.rng(4)) < 0.6] = 123
    ids[::17] = -1
    ids[5::19] = v + 3
    check_grad(ids, w, 8, 32, F32, 1.0, "hot token")


def test_grad_runs_of_exact_pieces():
    """Runs of 31, 32, 33, 64, 65 and 96 tokens side by side."""
    lens = [31, 32, 33, 64, 65, 96, 1, 32, 33]
    ids = torch.cat([torch.full((n,), 3 * i, dtype=torch.int32) for i, n in enumerate(lens)])
    ids = ids[torch.randperm(len(ids), generator=oh.rng(6))]
    w = table(30, 96, 6, 32, F16)
    check_grad(ids, w, 6, 32, F16, 1.0, "pieces")


def test_grad_no_tokens():
    w = table(12, 64, 4, 32, BF16)
    ids = torch.empty((0,), dtype=torch.int32, device=dev())
    ds, db = qp.qembedding_backward(ids, torch.empty((0, 64), dtype=torch.bfloat16, device=dev()),
                                    w[0].to(dev()), 4, 32)
    assert ds.shape == (12, 2) and not ds.any() and not db.any()


def test_grad_against_differences():
    """The lookup is linear in scales and biases: differences of the 64-bit form are exact."""
    v, k, bits, gs = 15, 96, 4, 32
    w = table(v, k, bits, gs, F32)
    ids = torch.randint(0, v, (40,), generator=oh.rng(7)).to(torch.int32)
    dout = oh.normal((40, k), 1.0, F32, oh.rng(8))
    got = qp.qembedding_backward(ids.to(dev()), dout.to(dev()), w[0].to(dev()), bits, gs, factor=3.0)
    q = oh.codes(w[0], bits)
    p = [w[1].double(), w[2].double()]

    def loss(s, b):
        W = q * s.repeat_interleave(gs, 1) + b.repeat_interleave(gs, 1)
        return float((dout.double() * 3.0 * W[ids.long()]).sum())

    for i in (0, 1):
        d = torch.randn(p[i].shape, generator=oh.rng(9 + i)).double()
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-3 * d, p[i] - 1e-3 * d
        fd = (loss(*hi) - loss(*lo)) / 2e-3
        mine = got[i].cpu().double()
        mag = float((dout.double().abs() * 3.0 * 15).sum())
        assert abs(float((mine * d).sum()) - fd) <= 1e-5 * mag, (i, float((mine * d).sum()), fd)


@pytest.mark.parametrize("v", [300, 2 ** 21 + 5])
@pytest.mark.parametrize("t", [111 * 2048, 111 * 2048 + 1, 113 * 2048 - 7, 2 ** 18 + 2049])
def test_grad_many_tokens(t, v):
    """On both sides of the number of sorted chunks from which runs are merged, with runs that
    are whole, short and odd in number; ids outside the table among them."""
    k = 32
    ids = torch.randint(-1, 301, (t,), generator=oh.rng(t)).to(torch.int32)
    if v > 300:
        ids[::1000] = v - 1
        ids[1::1000] = v
    log(f"embedding grad t={t} v={v} k={k}")
    check_grad(ids, table(v, k, 2, 32, F16), 2, 32, F16, 1.0, "many tokens")
