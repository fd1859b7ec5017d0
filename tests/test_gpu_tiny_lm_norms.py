"""examples/tiny_lm.py with norms: it trains and decodes, the same seed gives the same losses,
and its gradients are those of the same model in 64 bits, whose own agree with differences."""
from __future__ import annotations

import pytest
import torch

import ophelpers as oh
from qhelpers import log
from test_gpu_tiny_lm import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,gs,act,dtype", [
    (4, 32, "silu", torch.bfloat16), (6, 64, "gelu_tanh", torch.float16), (8, 128, "silu", torch.float32)])
def test_runs_and_repeats(bits, gs, act, dtype):
    lm = example()
    runs = []
    for _ in range(2):
        log(f"tiny model with norms: {bits} bits, groups of {gs}, {act}, {dtype}")
        model = lm.TinyLM(bits=bits, group_size=gs, act=act, dtype=dtype, norms=True)
        runs.append((lm.train(model, 12), lm.decode(model, ["the", "a tok"], 6, "abcdefghijklmnopqrstuvwxyz .")))
    assert runs[0] == runs[1]
    assert all(loss == loss and loss < 20 for loss in runs[0][0])
    assert [len(t) for t in runs[0][1]] == [9, 11]


def rms_norm(s, weight):
    return s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6) * weight


def loss64(model, ids, targets, params):
    """The mean loss in 64 bits; params: scales and biases of weights(), then the norms."""
    it = iter(params)

    def weight(w):
        s, b = next(it), next(it)
        return oh.codes(w[0].cpu(), model.bits) * s.repeat_interleave(model.gs, 1) + b.repeat_interleave(model.gs, 1)

    table, *rest = [weight(w) for w in model.weights()]
    norms = list(it)
    s = table[ids.long().cpu()] * model.factor
    a = rms_norm(s, norms[0])
    for i, w in enumerate(norms[1:]):
        gate, up, down = rest[3 * i:3 * i + 3]
        s = s + (torch.nn.functional.silu(a @ gate.t()) * (a @ up.t())) @ down.t()
        a = rms_norm(s, w)
    z = a @ rest[-1].t()
    return (torch.logsumexp(z, 1) - z.gather(1, targets.long().cpu()[:, None])[:, 0]).mean()


def test_gradients():
    """The fp32 model's gradients, tensor by tensor. Each comes out of at most eight products of up
    to 512 terms, whose roundings are 2^-24 of their terms and of random signs: about 8 sqrt(512)
    2^-24 = 1e-5 of a tensor's norm, 30 times that where sums cancel; a term left out or taken
    twice is some tenths."""
    lm = example()
    log("gradients of the tiny model with norms")
    model = lm.TinyLM(dtype=torch.float32, norms=True, seed=3)
    g = oh.rng(4)
    for t in model.norms:
        t += 0.2 * torch.randn(t.shape, generator=g).to(t.device)
    ids, targets = (torch.randint(0, lm.VOCAB, (70,), generator=g).to(torch.int32).cuda() for _ in range(2))
    loss, pairs, norms = model.loss_and_gradients(ids, targets)
    got = [t.cpu().double() for p in pairs for t in p] + [t.cpu().double() for t in norms]
    params = [t.cpu().double().requires_grad_() for w in model.weights() for t in w[1:]]
    params += [t.cpu().double().requires_grad_() for t in model.norms]
    want = loss64(model, ids, targets, params)
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-4
    for i, (a, p) in enumerate(zip(got, params)):
        assert a.shape == p.shape
        assert float((a - p.grad).norm()) <= 3e-4 * float(p.grad.norm()), i
    # Central differences of the 64-bit loss along one direction through all tensors; their error
    # falls with eps^2, and is a third of what twice the eps changes.
    direction = [torch.randn(p.shape, generator=g).double() * p.detach().abs().mean() for p in params]

    def slope(eps):
        up, down = ([p.detach() + sign * eps * d for p, d in zip(params, direction)] for sign in (1, -1))
        return float(loss64(model, ids, targets, up) - loss64(model, ids, targets, down)) / (2 * eps)

    inner = sum(float((a * d).sum()) for a, d in zip(got, direction))
    size = sum(float(p.grad.norm() * d.norm()) for p, d in zip(params, direction))
    fd, fd2 = slope(1e-4), slope(2e-4)
    assert abs(inner - fd) <= 3e-4 * size + abs(fd2 - fd) + 1e-8
