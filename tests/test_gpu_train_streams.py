"""The loss and the norms as a training step uses them together: the same bits eagerly, on a
stream of the caller's and from a captured graph, replayed several times with eager work and
synchronisations between the replays; two captured graphs over workspaces of their own; and
the whole step's gradients against the 64-bit chain's."""
from __future__ import annotations

import pytest
import torch

import weight_only_quantized_qgemv_amd as qp
import ophelpers as oh
from qhelpers import BF16, F32, TAU, dev, log

pytestmark = pytest.mark.gpu

BITS, GS, D, F, V = 4, 64, 256, 448, 1100


class Step:
    """Embedding, two blocks with norms around them, the loss, and all the gradients."""

    def __init__(self, rows=(1, 7, 40, 300), seed=17, dt=BF16):
        g = oh.rng(seed)
        self.dt, self.rows = dt, rows
        self.table, self.head = oh.weight(V, D, BITS, GS, dt, g), oh.weight(V, D, BITS, GS, dt, g)
        self.blocks = [(oh.weight(F, D, BITS, GS, dt, g), oh.weight(F, D, BITS, GS, dt, g), oh.weight(D, F, BITS, GS, dt, g))
                       for _ in range(2)]
        self.norms = [oh.normal((D,), 0.2, dt, g) + 1 for _ in range(3)]
        self.posts = [oh.normal((D,), 0.2, dt, g) + 1 for _ in range(2)]
        self.gates = [oh.normal((1, D), 0.5, dt, g) for _ in range(2)]
        self.ids = {m: torch.randint(0, V, (m,), generator=g).to(torch.int32) for m in rows}
        self.targets = {m: torch.randint(-1, V, (m,), generator=g).to(torch.int32) for m in rows}
        for name in ("table", "head"):
            setattr(self, name, oh.cuda(getattr(self, name)))
        self.blocks = [tuple(oh.cuda(w) for w in b) for b in self.blocks]
        for name in ("norms", "posts", "gates"):
            setattr(self, name, [t.to(dev()) for t in getattr(self, name)])
        for d in (self.ids, self.targets):
            for m in rows:
                d[m] = d[m].to(dev())
        self.dloss = {m: torch.full((m,), 1.0 / m, device=dev()) for m in rows}

    def step(self, m):
        q = (BITS, GS)
        s = qp.qembedding(self.ids[m], *self.table, *q, 16.0).float()     # the stream, in fp32
        s, a = qp.qblock_norm(s, weight=self.norms[0])
        kept, saved = [s], []
        for i, block in enumerate(self.blocks):
            keep = torch.empty((2, m, F), dtype=a.dtype, device=dev())
            y = qp.qffn(a, *block, *q, saved=keep)
            saved.append((a, keep, y))
            s, a = qp.qblock_norm(s, y, self.norms[i + 1], self.posts[i], self.gates[i], 0.5)
            kept.append(s)
        loss, lse = qp.qcross_entropy(a, self.targets[m], *self.head, *q)
        da, *grads = qp.qcross_entropy_backward(a, self.targets[m], lse, self.dloss[m], *self.head, *q)
        out, ds = [loss, lse, *kept, *grads], None
        for i in (1, 0):
            a, keep, y = saved[i]
            ds, dy, *more = qp.qblock_norm_backward(kept[i + 1], da, ds, y, self.norms[i + 1], self.posts[i], self.gates[i], 0.5)
            da, *pairs = qp.qffn_backward(a, dy, keep, *self.blocks[i], *q)
            out += [ds, *more, da, *(t for p in pairs for t in p)]
        ds, _, dw, _, _ = qp.qblock_norm_backward(kept[0], da, ds, weight=self.norms[0])
        return out + [ds, dw]

    def run(self):
        return [t for m in self.rows for t in self.step(m)]


def same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert oh.same_bits(x, y), f"output {i}"


def test_graph_replays_match_eager():
    log("graph capture of a training step")
    c, other = Step(), Step(seed=18)
    want, want2 = [t.clone() for t in c.run()], [t.clone() for t in other.run()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in (c, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            outs.append(s.run())
        graphs.append(g)
    for i in range(4):
        log(f"replay {i}")
        for t in outs[0] + outs[1]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        same(want, outs[0])
        same(want2, outs[1])
        same(want, c.run())


def test_on_another_stream_beside_eager_work():
    log("a training step on a side stream")
    c, other = Step(), Step(seed=18)
    want, want2 = c.run(), other.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    got2 = other.run()      # at the same time
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same(want, got)
    same(want2, got2)


def test_the_steps_gradients_against_64_bits():
    """fp32 throughout: TAU of the sum of magnitudes is far above what two blocks' fp32 sums lose;
    a gradient's magnitudes are taken as its own norm's share, 1e-4 of it (300 times what the
    chain's some 300 thousand additions of 2^-24 give at random)."""
    c = Step(rows=(23,), dt=F32)
    out = c.step(23)
    torch.cuda.synchronize()
    w64 = lambda w: oh.dense(tuple(t.cpu() for t in w), BITS, GS)   # noqa: E731
    norms, posts, gates = ([t.cpu().double().requires_grad_() for t in ts] for ts in (c.norms, c.posts, c.gates))
    s0 = (w64(c.table)[c.ids[23].cpu().long()] * 16.0).requires_grad_()
    norm = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w   # noqa: E731
    s, a = s0, norm(s0, norms[0])
    for i, block in enumerate(c.blocks):
        wg, wu, wd = (w64(w) for w in block)
        y = (torch.nn.functional.silu(a @ wg.t()) * (a @ wu.t())) @ wd.t()
        s = s + 0.5 * gates[i] * norm(y, posts[i])
        a = norm(s, norms[i + 1])
    t = c.targets[23].cpu().long()
    live = t >= 0
    z = a @ w64(c.head).t()
    loss = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    loss.mean().backward()

    def near(got, want, what):
        off = float((got.cpu().double() - want.detach()).norm() / want.detach().norm())
        assert off <= 1e-4, (what, off)

    near(out[0], loss, "loss")
    near(out[-2], s0.grad, "ds")
    near(out[-1], norms[0].grad, "dweight 0")
    at = 2 + 3 + 2   # loss, lse; three streams; the head's gradients
    for i in (1, 0):
        _, dweight, dpost, dgate = out[at:at + 4]
        near(dweight, norms[i + 1].grad, f"dweight {i + 1}")
        near(dpost, posts[i].grad, f"dpost {i}")
        near(dgate, gates[i].grad, f"dgate {i}")
        at += 4 + 1 + 6
