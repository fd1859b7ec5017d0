"""qblock_norm and its backward pass with the most rows that they take, 2^22: narrow rows and,
forward, rows of 512 threads each. Rows are compared with calls of a few of them."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, dev, log

pytestmark = pytest.mark.gpu

M = 1 << 22


def rows(d, sigma, g):
    """2^22 rows, repeating after 4099 (a prime) with their elements turned by one."""
    part = torch.randn((4099, d), generator=g, device=dev()) * sigma
    out = torch.empty((M, d), dtype=torch.bfloat16, device=dev())
    for at in range(0, M, 4099):
        n = min(4099, M - at)
        out[at:at + n] = part[:n].roll(at // 4099, 1)
    return out


def test_narrow_rows():
    log(f"norm of {M} rows of 12")
    d, g = 12, torch.Generator(device="cuda").manual_seed(1)
    x, y, da, ds = (rows(d, v, g) for v in (3.0, 2.0, 0.1, 0.1))
    w, post, gate = ((torch.randn(s, generator=g, device=dev()) * 0.2 + 1).bfloat16() for s in ((d,), (d,), (1, d)))
    s, a = qp.qblock_norm(x, y, w, post, gate, 0.5)
    dx, dy, dw, dp, dg = qp.qblock_norm_backward(s, da, ds, y, w, post, gate, 0.5)
    for at in (0, M // 2 + 1, M - 4):
        cut = slice(at, at + 4)
        s1, a1 = qp.qblock_norm(x[cut], y[cut], w, post, gate, 0.5)
        dx1, dy1, *_ = qp.qblock_norm_backward(s[cut], da[cut], ds[cut], y[cut], w, post, gate, 0.5)
        assert all(oh.same_bits(p[cut], q) for p, q in ((s, s1), (a, a1), (dx, dx1), (dy, dy1))), at
    # dweight in 64 bits: 2^22 rows over 2048 blocks, then their sums.
    sd = s.double()
    terms = da.double() * sd * torch.rsqrt((sd * sd).mean(1, keepdim=True) + 1e-6)
    want, size = terms.sum(0).cpu(), terms.abs().sum(0).cpu()
    oh.check(dw, want, oh.gamma(M // 2048 + 2048 + d) * size + oh.half_ulp(want, BF16), "dweight")


def test_wide_rows():
    if torch.cuda.get_device_properties(0).total_memory < 100 * 2 ** 30:
        pytest.skip("needs 100 GiB of GPU memory")
    d, g = 2056, torch.Generator(device="cuda").manual_seed(2)
    log(f"norm of {M} rows of {d}")
    x = rows(d, 3.0, g)
    w = (torch.randn(d, generator=g, device=dev()) * 0.2 + 1).bfloat16()
    _, a = qp.qblock_norm(x, weight=w)
    for at in (0, M // 2 + 1, M - 4):
        _, a1 = qp.qblock_norm(x[at:at + 4], weight=w)
        assert oh.same_bits(a[at:at + 4], a1), at
