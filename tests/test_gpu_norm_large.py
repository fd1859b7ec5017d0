"""qblock_norm and its backward pass on tensors of more than 2^31 elements: each row is the same
bits as in a call of a few rows, and the weights' gradients are the rows' sums."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F16, F32, dev, log
from test_gpu_norm import Case, run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d,dt,sdt,post,gates,pre,y", [
    (700, 8200, BF16, BF16, True, 1, True, True), (700, 8208, F16, F32, True, 2, True, True),
    (1100, 8193, F32, F32, True, 1, True, True), (520, 16384, BF16, F32, False, 1, True, True),
    (800, 8200, BF16, BF16, False, 0, True, True), (800, 8200, BF16, BF16, False, 0, True, False),
    (800, 8200, BF16, F32, True, 4, False, True), (258, 8200, F16, F16, True, 129, True, True)])
def test_wide_rows_several_to_a_block(m, d, dt, sdt, post, gates, pre, y):
    """Three rows at a time, of which the last group has one, two or three."""
    run_and_check(Case(m, d, dt, sdt, post, gates, pre, y=y), "wide")


@pytest.mark.parametrize("m,d", [((1 << 20) + 3, 4096), ((1 << 17) + 5, 16384)])
def test_more_than_2_31_elements(m, d):
    if torch.cuda.get_device_properties(0).total_memory < 80 * 2 ** 30:
        pytest.skip("needs 80 GiB of GPU memory")
    log(f"norm of {m} rows of {d}")
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(sigma):
        out = torch.empty((m, d), dtype=torch.bfloat16, device=dev())
        part = torch.randn((4099, d), generator=g, device=dev()) * sigma     # (a prime: no row meets itself)
        for at in range(0, m, 4099):
            n = min(4099, m - at)
            out[at:at + n] = part[:n].roll(at // 4099, 1)
        return out

    x, y = rows(3.0), rows(2.0)
    w, post, gate = ((torch.randn(s, generator=g, device=dev()) * 0.2 + 1).bfloat16() for s in ((d,), (d,), (1, d)))
    factor = 0.5
    s, a = qp.qblock_norm(x, y, w, post, gate, factor)
    picks = [0, 2 ** 31 // d - 2, 2 ** 31 // d + 1, m - 4]
    for at in picks:
        s1, a1 = qp.qblock_norm(x[at:at + 4], y[at:at + 4], w, post, gate, factor)
        assert oh.same_bits(s[at:at + 4], s1) and oh.same_bits(a[at:at + 4], a1), at
    del x, a
    da, ds = rows(0.1), rows(0.1)
    dx, dy, dw, dp, dg = qp.qblock_norm_backward(s, da, ds, y, w, post, gate, factor)
    for at in picks:
        cut = [t[at:at + 4] for t in (s, da, ds, y)]
        dx1, dy1, *_ = qp.qblock_norm_backward(*cut, w, post, gate, factor)
        assert oh.same_bits(dx[at:at + 4], dx1) and oh.same_bits(dy[at:at + 4], dy1), at
    # dweight, in 64 bits: a column is summed over 512 blocks of m / 512 rows at most, each term a
    # few roundings.
    want, size = (torch.zeros(d, dtype=torch.float64, device=dev()) for _ in range(2))
    for at in range(0, m, 16384):
        sd, dd = s[at:at + 16384].double(), da[at:at + 16384].double()
        terms = dd * sd * torch.rsqrt((sd * sd).mean(1, keepdim=True) + 1e-6)
        want += terms.sum(0)
        size += terms.abs().sum(0)
    n = m // 256 + 512 + d      # (a block may take two shares; d: the row's own mean)
    want, size = want.cpu(), size.cpu()
    oh.check(dw, want, oh.gamma(n) * size + oh.half_ulp(want, BF16), "dweight")
