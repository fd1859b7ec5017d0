"""Calls of more threads than one grid dimension takes (2^32), in sizes that fit the GPU."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import F16, dev, log

pytestmark = pytest.mark.gpu


def need(gib):
    if torch.cuda.get_device_properties(0).total_memory < gib * 2 ** 30 * 1.1:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_embedding_of_more_than_2_24_tokens():
    """2^24 tokens of 2048 columns, 64 GiB: compared slice by slice with calls of a few tokens."""
    need(80)
    t, v, k, bits, gs = 2 ** 24 + 5, 97, 2048, 2, 128
    log(f"lookup of {t} tokens of {k}")
    w = oh.cuda(oh.weight(v, k, bits, gs, F16, oh.rng(1)))
    ids = (torch.arange(t, dtype=torch.int64, device=dev()) * 31 % (v + 1)).to(torch.int32)   # id v: zeros
    rows = qp.qembedding(torch.arange(v + 1, dtype=torch.int32, device=dev()), *w, bits, gs, 2.0)
    out = qp.qembedding(ids, *w, bits, gs, 2.0)
    step = 2 ** 20
    for at in range(0, t, step):
        part = ids[at:at + step].long()
        assert torch.equal(out[at:at + step].view(torch.int16), rows.view(torch.int16)[part]), at
    del out


@pytest.mark.parametrize("same", [False, True])
def test_embedding_gradient_of_2_27_tokens(same):
    """2^27 + 2049 tokens: sums of ones, exact in fp32 below 2^24 each. With one id for most
    tokens a single run crosses most windows."""
    need(60)
    t, v, k, bits, gs = 2 ** 27 + 2049, 4001, 32, 8, 32
    log(f"embedding gradient of {t} tokens, one id: {same}")
    g = torch.Generator(device="cuda").manual_seed(5)
    wq = torch.zeros((v, k * bits // 32), dtype=torch.int32, device=dev())
    wq[:, 0] = 3                                  # column 0 has code 3, the others 0
    ids = torch.randint(-1, v + 1, (t,), generator=g, device=dev(), dtype=torch.int32)
    if same:
        ids[torch.rand(t, generator=g, device=dev()) < 0.9] = 77
    live = (ids >= 0) & (ids < v)
    count = torch.bincount(ids[live].long(), minlength=v).double()
    # Every token adds 2^-10 at column 0: sums of up to 2^27 tokens, fp32 partial sums in order.
    dout = torch.zeros((t, k), dtype=torch.bfloat16, device=dev())
    dout[:, 0] = 2.0 ** -10
    ds, db = qp.qembedding_backward(ids, dout, wq, bits, gs)
    for got, want in ((ds, 3 * count * 2.0 ** -10), (db, count * 2.0 ** -10)):
        bound = want * 2.0 ** -8 + want * oh.gamma(64)   # half an ulp of bf16, and partial sums of windows
        assert ((got[:, 0].double() - want).abs() <= bound).all()


def test_logits_of_more_than_2_23_rows():
    rows, v = 2 ** 23 + 3, 32
    log(f"logits of {rows} rows of {v}")
    z = torch.arange(rows * v, device=dev(), dtype=torch.int32).remainder(251).to(torch.bfloat16).view(rows, v)
    mask = torch.tensor([[0x7FFFFFFE]], dtype=torch.int32, device=dev())
    out = qp.qlogits_adjust(z, mask=mask)
    assert torch.equal(out[:, 1:31], z[:, 1:31])
    assert (out[:, 0] == float("-inf")).all() and (out[:, 31] == float("-inf")).all()


def big_weight(n, k, gs, dt, entries):
    """8-bit weights [n, k] of 2 GiB and more on the device: scale 1, bias 0, entries
    (row, column, code)."""
    q = torch.zeros((n, k), dtype=torch.uint8, device=dev())
    for r, c, code in entries:
        q[r, c] = code
    one = torch.ones((n, k // gs), dtype=dt, device=dev())
    return q.view(torch.int32), one, torch.zeros_like(one)


@pytest.mark.parametrize("m", [1, 3, 20])
def test_block_of_weights_of_2_gib(m):
    """Weights past the 32-bit offsets of the tile and skinny kernels: exact numbers in the last
    rows and columns (bf16: g = 257, u = 129, h = 33153, which rounds to 33152)."""
    need(20)
    d, f, gs, dt = 32768, 65600, 32, torch.bfloat16
    log(f"block of 2 GiB weights, {m} rows")
    x = torch.zeros((m, d), dtype=dt, device=dev())
    x[:, d - 1] = x[:, d - 2] = 1
    gate = big_weight(f, d, gs, dt, [(f - 1, d - 1, 255), (f - 1, d - 2, 2)])
    up = big_weight(f, d, gs, dt, [(f - 1, d - 1, 127), (f - 1, d - 2, 2)])
    down = big_weight(d, f, gs, dt, [(d - 1, f - 1, 1)])
    saved = torch.empty((2, m, f), dtype=dt, device=dev())
    for kept in (None, saved):
        y = qp.qffn(x, gate, up, down, 8, gs, saved=kept)
        torch.cuda.synchronize()
        assert (y[:, d - 1] == 33152).all() and not y[:, :d - 1].any()
    assert (saved[0, :, f - 1] == 256).all() and (saved[1, :, f - 1] == 129).all()
    assert not saved[:, :, :f - 1].any()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_and_lookup_of_a_weight_of_2_gib(dt):
    need(20)
    m, n, k, gs = 3, 65600, 32768, 32
    log(f"gradients of a 2 GiB weight, {dt}")
    w = big_weight(n, k, gs, dt, [(n - 1, k - 1, 255), (n - 1, 0, 3), (n - 2, 5, 7)])
    x, dy = (torch.zeros((m, c), dtype=dt, device=dev()) for c in (k, n))
    x[2, k - 1], x[2, 0], dy[2, n - 1] = 2, 1, 4
    dx, ds, db = qp.qmatmul_backward(x, dy, *w, 8, gs)
    torch.cuda.synchronize()
    want = torch.zeros_like(dx)
    want[2, k - 1], want[2, 0] = 1020, 12         # 4 times the last weight row
    assert torch.equal(dx, want)
    # dW's last row is 4 x[2]: 8 in the last column, 4 in the first.
    for got, first, last in ((ds, 4 * 3, 8 * 255), (db, 4, 8)):
        assert float(got[n - 1, 0]) == first and float(got[n - 1, -1]) == last
        assert not got[:n - 1].any() and not got[n - 1, 1:-1].any()
    ids = torch.tensor([n - 1, 0, n - 2], dtype=torch.int32, device=dev())
    rows = qp.qembedding(ids, *w, 8, gs)
    assert float(rows[0, k - 1]) == 255 and float(rows[0, 0]) == 3 and float(rows[2, 5]) == 7
    assert int((rows != 0).sum()) == 3
    ds, db = qp.qembedding_backward(ids, x, w[0], 8, gs)
    torch.cuda.synchronize()
    assert float(ds[n - 2, 0]) == 0 and float(db[n - 2, 0]) == 1 and float(db[n - 2, -1]) == 2
    assert float(ds[n - 1, 0]) == 0 and not db[n - 1].any() and not db[:n - 2].any()


def test_block_backward_past_2_gib():
    """dg, du and h of more than 2 GiB each, every row the same: exact numbers everywhere."""
    need(30)
    m, d, f, gs, dt = 70000, 64, 16384, 64, torch.bfloat16
    log(f"block backward, {m} rows of {f}")
    gate = big_weight(f, d, gs, dt, [(f - 1, d - 1, 1)])
    up = big_weight(f, d, gs, dt, [(f - 1, 0, 1)])
    down = big_weight(d, f, gs, dt, [(5, f - 1, 1)])
    x, dy = (torch.zeros((m, d), dtype=dt, device=dev()) for _ in range(2))
    x[:, 3], dy[:, 5] = 1, 1
    saved = torch.zeros((2, m, f), dtype=dt, device=dev())
    saved[0, :, f - 1], saved[1, :, f - 1] = 256, 129     # act(256) = 256, act' = 1
    dx, dgate, dup, ddown = qp.qffn_backward(x, dy, saved, gate, up, down, 8, gs)
    torch.cuda.synchronize()
    want = torch.zeros((d,), dtype=dt, device=dev())
    want[d - 1], want[0] = 129, 256               # dg Wg + du Wu
    assert torch.equal(dx, want.expand(m, d))
    # Sums over the rows of dg, du and h, exact in fp32, at code 0 (and, down, code 1).
    total = lambda v: float(torch.tensor(float(v * m)).to(dt))  # noqa: E731
    for (ds, db), value in ((dgate, 129), (dup, 256)):
        assert not ds.any() and float(db[f - 1, 0]) == total(value) and not db[:f - 1].any()
    ds, db = ddown
    h = 256 * 129                                 # 33024, exact in eight bits
    assert float(ds[5, -1]) == total(h) and float(db[5, -1]) == total(h)
    assert int((ds != 0).sum()) == 1 and int((db != 0).sum()) == 1
