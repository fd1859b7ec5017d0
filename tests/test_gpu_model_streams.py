"""The operators around the products under HIP graph capture and on a stream of
the caller's: a captured sequence, replayed several times with eager work and
synchronisations between the replays, and the same calls on a side stream give
the eager calls' bits. The library allocates nothing and records no memset."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
from ophelpers import cuda, normal, rng, weight
from qhelpers import BF16, dev, log

pytestmark = pytest.mark.gpu

BITS, GS, D, F, V = 4, 64, 256, 448, 1000
ROWS = (1, 2, 12, 40)          # each forward kernel
BACK = (40, 300)               # one tile and several


class Calls:
    """Inputs, outputs' buffers and one run of every operator."""

    def __init__(self):
        g = rng(71)
        self.gate, self.up = (cuda(weight(F, D, BITS, GS, BF16, g)) for _ in range(2))
        self.down = cuda(weight(D, F, BITS, GS, BF16, g))
        self.table = cuda(weight(V, D, BITS, GS, BF16, g))
        self.odd = cuda(weight(203, D, BITS, GS, BF16, g))      # rows of dy that are padded
        self.x = {m: cuda(normal((m, D), 1.0, BF16, g)) for m in (*ROWS, *BACK)}
        self.dy = {m: cuda(normal((m, D), 1.0, BF16, g)) for m in BACK}
        self.dodd = {m: cuda(normal((m, 203), 1.0, BF16, g)) for m in BACK}
        self.ids = torch.randint(-1, V + 1, (2500,), generator=g).to(torch.int32).to(dev())
        self.dout = cuda(normal((2500, D), 1.0, BF16, g))
        self.logits = cuda(normal((3, V), 2.0, BF16, g))
        self.hist = torch.randint(0, V, (90,), generator=g).to(torch.int32).to(dev())
        self.offs = torch.tensor([0, 30, 30, 90], dtype=torch.int32, device=dev())
        self.pen = torch.tensor([1.1, 1.2, 1.3], device=dev())
        self.mask = torch.randint(-2 ** 31, 2 ** 31, (3, (V + 31) // 32), generator=g).to(torch.int32).to(dev())

    def run(self):
        w = (self.gate, self.up, self.down, BITS, GS)
        out = [qp.qffn(self.x[m], *w) for m in ROWS]
        for m in BACK:
            saved = torch.empty((2, m, F), dtype=torch.bfloat16, device=dev())
            out.append(qp.qffn(self.x[m], *w, saved=saved))
            dx, *pairs = qp.qffn_backward(self.x[m], self.dy[m], saved, *w)
            out += [saved, dx, *(t for p in pairs for t in p)]
            out += qp.qmatmul_backward(self.x[m], self.dodd[m], *self.odd, BITS, GS)
        out.append(qp.qembedding(self.ids, *self.table, BITS, GS, 2.0))
        out += qp.qembedding_backward(self.ids, self.dout, self.table[0], BITS, GS, 2.0)
        out.append(qp.qlogits_adjust(self.logits, self.hist, self.offs, None, self.pen, self.pen, self.pen,
                                     mask=self.mask))
        return out


def same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16)), f"output {i}"


def test_graph_replays_match_eager():
    log("graph capture of the operators around the products")
    c = Calls()
    want = [t.clone() for t in c.run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = c.run()
    for i in range(4):
        log(f"replay {i}")
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(want, got)
        same(want, c.run())


def test_on_another_stream():
    log("the operators around the products on a side stream")
    c = Calls()
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same(want, got)
