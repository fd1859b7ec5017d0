"""GPU parity of qlogits_adjust with its 64-bit form.

Bound: at most six fp32 roundings (the division or product by the repetition, the
frequency's product and the three sums) of the largest magnitude that occurs on the
way, and half an ulp of the result; -inf, infinities and NaN have to agree exactly.
"""
from __future__ import annotations

import math

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, TORCH_DT, dev, log

pytestmark = pytest.mark.gpu


def reference(z, hists, prompts, rep, freq, pres, bias, mask):
    """Row by row, token by token; also the largest magnitude on the way."""
    out, mag = z.double().clone(), z.double().abs()
    rows, v = z.shape
    for r in range(rows):
        counts = {}
        for i, t in enumerate(hists[r]):
            if 0 <= t < v:
                counts[t] = counts.get(t, 0) + (i >= prompts[r])
        for t, c in counts.items():
            x = float(out[r, t])
            x = x / rep[r] if x > 0 else x * rep[r]
            m = max(abs(x), float(mag[r, t]))
            if c:
                m += abs(freq[r] * c) + abs(pres[r])
                x = x - freq[r] * c - pres[r]
            out[r, t], mag[r, t] = x, m
        if bias is not None:
            for t, b in dict(bias[r]).items():   # the last entry of a token counts
                if 0 <= t < v:
                    out[r, t] += b
                    mag[r, t] += abs(b)
        if mask is not None:
            out[r, ~mask[r]] = -math.inf
            mag[r, ~mask[r]] = 0.0
    return out, mag


def pack(mask):
    rows, v = mask.shape
    words = (v + 31) // 32
    bits = torch.zeros((rows, words * 32), dtype=torch.int64)
    bits[:, :v] = mask.long()
    w = (bits.reshape(rows, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def ragged(lists, dtype):
    off = torch.tensor([0] + [len(x) for x in lists]).cumsum(0).to(torch.int32)
    return torch.tensor([t for x in lists for t in x], dtype=dtype), off


def f32(v):
    return [float(t) for t in torch.tensor(v, dtype=torch.float32)]


def compare(got, ref, mag, dt, what):
    got = got.cpu().double()
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    inf = odd & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), what
    ok = ~odd
    bound = 6 * 2.0 ** -24 * mag + oh.half_ulp(ref, dt)
    bad = (got - ref).abs()[ok] > bound[ok]
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float((got - ref).abs()[ok].max()):.3e}"


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("rows,v,pad", [(1, 1, 0), (1, 31, 0), (3, 33, 1), (2, 1000, 24), (4, 4095, 0), (2, 4096, 0),
                                        (2, 4097, 7), (5, 12345, 3), (1, 70001, 0)])
@pytest.mark.parametrize("full", [False, True])
def test_all_controls(rows, v, pad, dt, full):
    g = oh.rng(oh.seed_of(rows, v, pad, dt))
    log(f"logits rows={rows} v={v} pad={pad} dt={dt} full={full}")
    z = (torch.randn((rows, v + pad), generator=g) * 4).to(TORCH_DT[dt])
    lens = torch.randint(0, 300, (rows,), generator=g).tolist()
    lens[-1] = 0
    # Tokens cluster (counts above one) and some lie outside the vocabulary.
    hists = [torch.randint(-2, max(min(v, 40), 1) + 2, (n,), generator=g).tolist() for n in lens]
    prompts = [n // 3 for n in lens]
    rep, freq, pres = (f32((torch.rand(rows, generator=g) + o).tolist()) for o in (0.7, -0.2, -0.4))
    bias = mask = None
    kw = {}
    if full:
        bias = [[(int(t), float(b)) for t, b in zip(torch.randint(-1, v + 1, (9,), generator=g),
                                                    torch.randn(9, generator=g))] for _ in range(rows)]
        bias[0] += [(0, 1.0), (0, -2.5)]
        mask = torch.rand((rows, v), generator=g) < 0.5
        mask[rows - 1] = False                     # a row that may say nothing
        ids, off = ragged([[t for t, _ in b] for b in bias], torch.int32)
        vals, _ = ragged([[b for _, b in x] for x in bias], torch.float32)
        kw = {"bias": (ids.to(dev()), vals.to(dev()), off.to(dev())), "mask": pack(mask).to(dev())}
    hist, hoff = ragged(hists, torch.int32)
    t = lambda a, d=torch.float32: torch.tensor(a, dtype=d).to(dev())  # noqa: E731
    zd = z.to(dev())[:, :v]
    args = dict(history=hist.to(dev()), offsets=hoff.to(dev()), prompt_lens=t(prompts, torch.int32),
                repetition=t(rep), frequency=t(freq), presence=t(pres), **kw)
    got = qp.qlogits_adjust(zd, **args)
    ref, mag = reference(z[:, :v], hists, prompts, rep, freq, pres, bias, mask)
    compare(got, ref, mag, dt, "all controls")
    # In place, the padding untouched.
    whole = z.to(dev())
    view = whole[:, :v]
    qp.qlogits_adjust(view, out=view, **args)
    assert oh.same_bits(view, got) and oh.same_bits(whole[:, v:], z[:, v:].to(dev()))


def test_single_controls_and_none():
    g = oh.rng(3)
    z = torch.randn((3, 500), generator=g).to(torch.bfloat16)
    zd = z.to(dev())
    assert oh.same_bits(qp.qlogits_adjust(zd), zd)
    hists = [[1, 2, 2, 2], [], [499, 0, 0]]
    hist, off = (x.to(dev()) for x in ragged(hists, torch.int32))
    ones, zeros = [1.0] * 3, [0.0] * 3
    some = f32([1.2, 1.3, 0.9])
    dv = torch.tensor(some).to(dev())
    for name, r, f, p in (("repetition", some, zeros, zeros), ("frequency", ones, some, zeros),
                          ("presence", ones, zeros, some)):
        got = qp.qlogits_adjust(zd, history=hist, offsets=off, **{name: dv})
        ref, mag = reference(z, hists, [0, 0, 0], r, f, p, None, None)
        compare(got, ref, mag, BF16, name)
    mask = torch.rand((1, 500), generator=g) < 0.3
    got = qp.qlogits_adjust(zd, mask=pack(mask).to(dev()))   # one mask for all rows
    ref, mag = reference(z, [[]] * 3, [0] * 3, ones, zeros, zeros, None, mask.expand(3, 500))
    compare(got, ref, mag, BF16, "shared mask")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_infinities_nan_and_lowest_values(dt):
    z = torch.zeros((2, 64)).to(TORCH_DT[dt])
    lowest = torch.finfo(TORCH_DT[dt]).min
    z[:, :8] = torch.tensor([math.inf, -math.inf, math.nan, lowest, -lowest, -0.0, 1e-30, -1e-30]).to(z.dtype)
    z[:, 8:16] = z[:, :8]
    mask = torch.ones((2, 64), dtype=torch.bool)
    mask[:, 8:16] = False                         # the same values in masked places
    hists = [list(range(16)), []]
    hist, off = (x.to(dev()) for x in ragged(hists, torch.int32))
    rep = torch.tensor([1.5, 1.5]).to(dev())
    got = qp.qlogits_adjust(z.to(dev()), history=hist, offsets=off, repetition=rep, mask=pack(mask).to(dev()))
    ref, mag = reference(z, hists, [0, 0], [1.5, 1.5], [0, 0], [0, 0], None, mask)
    if dt == BF16 or dt == F32:                   # lowest * 1.5 leaves the type
        ref[0, 3] = -math.inf
    compare(got, ref, torch.where(torch.isfinite(ref), mag, 0 * mag), dt, "special values")
    assert torch.isinf(got[:, 8:16]).all() and (got[:, 8:16] < 0).all()


def test_long_history_and_offsets_are_held_inside():
    v, n = 3000, 20000
    g = oh.rng(5)
    z = torch.randn((2, v), generator=g)
    h = torch.randint(0, v, (n,), generator=g).to(torch.int32)
    hists = [h[:15000].tolist(), h[15000:].tolist()]
    off = torch.tensor([0, 15000, n], dtype=torch.int32)
    freq = torch.tensor([0.25, 0.5])
    got = qp.qlogits_adjust(z.to(dev()), history=h.to(dev()), offsets=off.to(dev()), frequency=freq.to(dev()))
    ref, mag = reference(z, hists, [0, 0], [1.0] * 2, [0.25, 0.5], [0.0] * 2, None, None)
    compare(got, ref, mag, F32, "long history")
    # Offsets before the first and past the last token reach no further than the tokens.
    wild = torch.tensor([-50, 15000, n + 1000], dtype=torch.int32)
    assert oh.same_bits(got, qp.qlogits_adjust(z.to(dev()), history=h.to(dev()), offsets=wild.to(dev()),
                                               frequency=freq.to(dev())))


def test_far_offsets_are_held_inside():
    """Starts and ends near the ends of 32 bits, of tokens and of biases: a row whose offsets
    leave nothing inside is an empty one, and a start below zero is zero."""
    v, n, top = 600, 900, 2 ** 31 - 1
    g = oh.rng(6)
    z = torch.randn((6, v), generator=g)
    h = torch.randint(0, v, (n,), generator=g).to(torch.int32)
    # Offsets of row r are off[r] and off[r + 1].
    off = [top, top - 5, top - 1000, -2 ** 31, 40, top, top - 511]
    cut = [(min(max(a, 0), n), min(max(b, 0), n)) for a, b in zip(off, off[1:])]
    hists = [h[a:b].tolist() for a, b in cut]
    assert [len(x) for x in hists] == [0, 0, 0, 40, 860, 0]
    rep = f32([1.1, 1.2, 1.3, 1.4, 1.5, 1.6])
    bias = torch.randn(n, generator=g)
    biases = [list(zip(h[a:b].tolist(), bias[a:b].tolist())) for a, b in cut]
    offs = torch.tensor(off, dtype=torch.int32).to(dev())
    log("logits: offsets near the ends of 32 bits")
    got = qp.qlogits_adjust(z.to(dev()), history=h.to(dev()), offsets=offs,
                            prompt_lens=torch.tensor([top, -2 ** 31, 0, 7, top, 5], dtype=torch.int32).to(dev()),
                            repetition=torch.tensor(rep).to(dev()), frequency=torch.tensor([0.25] * 6).to(dev()),
                            bias=(h.to(dev()), bias.to(dev()), offs))
    ref, mag = reference(z, hists, [top, 0, 0, 7, top, 5], rep, [0.25] * 6, [0.0] * 6, biases, None)
    compare(got, ref, mag, F32, "far offsets")
