"""Plain 64-bit forms of the operators around the products, on the CPU, and the
error terms their tests add up.

A weight is (wq, scales, biases) on the CPU, w = q * s + b. Error terms:

* TAU * S for a product with a dequantized weight, S the sum of the products'
  magnitudes (qhelpers: the weight's rounding to 16 bits where the matrix
  cores take it, and fp32 accumulation);
* gamma(n) * S for a sum of n exact products in fp32 (n roundings of 2^-24,
  and the split sums' and the group sums' few more);
* half a unit in the last place of each rounding to the operator's type.
"""
from __future__ import annotations

import math

import torch

from qhelpers import F16, F32, HALF_SUBNORMAL, HALF_ULP, TORCH_DT, dev

DTYPES = {"f32": F32, "f16": F16, "bf16": 2}


def gamma(n: int) -> float:
    return (n + 64) * 2.0 ** -24


def half_ulp(v: torch.Tensor, dt: int) -> torch.Tensor:
    return torch.clamp(v.abs() * HALF_ULP[dt], min=HALF_SUBNORMAL[dt])


def rng(seed: int) -> torch.Generator:
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(shape, sigma, dt, g):
    return (torch.randn(shape, generator=g) * sigma).to(TORCH_DT[dt])


def weight(n, k, bits, gs, dt, g):
    """Random words (every code occurs) with scales and biases of both signs of imbalance."""
    wq = torch.randint(-2 ** 31, 2 ** 31, (n, k * bits // 32), generator=g).to(torch.int32)
    top = 2 ** bits - 1
    s = (torch.rand((n, k // gs), generator=g) + 0.5) * (3.0 / math.sqrt(k) / top)
    b = -s * top * torch.rand((n, k // gs), generator=g)
    return wq, s.to(TORCH_DT[dt]), b.to(TORCH_DT[dt])


def cuda(w):
    return tuple(t.to(dev()) for t in w) if isinstance(w, tuple) else w.to(dev())


def codes(wq, bits):
    """Codes of packed rows in fp64, from the rows' bits."""
    n = wq.shape[0]
    bit = (wq[:, :, None] >> torch.arange(32, dtype=torch.int32)) & 1
    stream = bit.reshape(n, -1, bits).double()
    return (stream * (2.0 ** torch.arange(bits).double())).sum(-1)


def spread(t, gs):
    return t.double().repeat_interleave(gs, dim=1)


def dense(w, bits, gs):
    wq, s, b = w
    return codes(wq, bits) * spread(s, gs) + spread(b, gs)


def group_sums(w, dW, bits, gs):
    """(dscales, dbiases) of the weight whose dense gradient is dW."""
    n, k = dW.shape
    q = codes(w[0], bits)
    return (dW * q).reshape(n, k // gs, gs).sum(-1), dW.reshape(n, k // gs, gs).sum(-1)


def act(z, name):
    """Activation and derivative, and the magnitude of the derivative's terms."""
    if name == "silu":
        p, dp = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        p, dp = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)
    s, t = torch.sigmoid(p), torch.sigmoid(-p)
    return z * s, s + z * s * t * dp, s + (z * s * t * dp).abs()


def check(y, ref, bound, what):
    y = y.detach().cpu().double()
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    err = (y - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err - bound, torch.full_like(err, -math.inf))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{y.flatten()[i]:.6e}, ref {ref.flatten()[i]:.6e}, err "
                             f"{err.flatten()[i]:.3e}, bound {bound.flatten()[i]:.3e}")


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def seed_of(*a) -> int:
    return sum(
        (i + 1) * sum(ord(c) for c in str(x)) for i, x in enumerate(a))
