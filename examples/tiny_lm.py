"""A small next-byte model on packed weights: trained, then decoded.

    python examples/tiny_lm.py [--steps N] [--bits B] [--seed S] [--norms]

The model is an embedding table, gated feed-forward blocks with residual
connections and an output head, every weight packed. Training keeps the codes
as they are and moves the scales and biases: forward (qembedding, qffn,
qmatmul), a cross entropy, then the backward passes (qmatmul_backward,
qffn_backward, qembedding_backward) and one Adam step over fp32 copies. With
--norms, each block's output goes through qblock_norm (the residual sum and the
norm before the next block, its weights trained too), and the loss and its
gradients come from qcross_entropy, without logits.
Decoding takes one token per sequence and step: the same forward at a few rows,
then qlogits_adjust (penalties from each sequence's own tokens, a mask of the
bytes that may appear) and the largest logit.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_qgemv_amd as qp   # noqa: E402

TEXT = ("the cache holds the keys and the values of the tokens seen so far. "
        "a router sends each token to its experts. the loss falls, step by step. ") * 40
VOCAB = 256


class TinyLM:
    def __init__(self, bits=4, group_size=32, d_model=256, d_ff=512, layers=2, act="silu",
                 dtype=torch.bfloat16, seed=0, norms=False):
        self.bits, self.gs, self.act, self.dtype = bits, group_size, act, dtype
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5
            return qp.qpack_quantize(w, bits, group_size, sb_dtype=dtype)

        self.table = weight(VOCAB, d_model)
        self.blocks = [(weight(d_ff, d_model), weight(d_ff, d_model), weight(d_model, d_ff))
                       for _ in range(layers)]
        self.head = weight(VOCAB, d_model)
        self.factor = d_model ** 0.5
        self.norms = [torch.ones(d_model, dtype=dtype, device="cuda") for _ in range(layers + 1)] if norms else []

    def weights(self):
        return [self.table, *(w for b in self.blocks for w in b), self.head]

    def forward(self, ids, keep=None):
        """Logits [tokens, VOCAB] of ids [tokens]; `keep`, a list, receives what backward() needs."""
        if self.norms:
            return qp.qmatmul(self.normed(ids), *self.head, self.bits, self.gs)
        x = qp.qembedding(ids, *self.table, self.bits, self.gs, self.factor)
        for block in self.blocks:
            saved = None
            if keep is not None:
                saved = torch.empty((2, x.shape[0], block[0][0].shape[0]), dtype=x.dtype, device=x.device)
                keep.append((x, saved))
            x = x + qp.qffn(x, *block, self.bits, self.gs, self.act, saved=saved)
        if keep is not None:
            keep.append(x)
        return qp.qmatmul(x, *self.head, self.bits, self.gs)

    def backward(self, ids, keep, dlogits):
        """Gradients (dscales, dbiases) in the order of weights()."""
        dx, ds, db = qp.qmatmul_backward(keep.pop(), dlogits, *self.head, self.bits, self.gs)
        grads = [(ds, db)]
        for block in reversed(self.blocks):
            x, saved = keep.pop()
            dxb, *pairs = qp.qffn_backward(x, dx, saved, *block, self.bits, self.gs, self.act)
            grads = [*pairs, *grads]
            dx = dx + dxb
        return [qp.qembedding_backward(ids, dx, self.table[0], self.bits, self.gs, self.factor), *grads]

    def normed(self, ids, keep=None):
        """The head's input, of a model with norms: one before each block and one before the head."""
        s, a = qp.qblock_norm(qp.qembedding(ids, *self.table, self.bits, self.gs, self.factor), weight=self.norms[0])
        for block, weight in zip(self.blocks, self.norms[1:]):
            saved = None
            if keep is not None:
                saved = torch.empty((2, a.shape[0], block[0][0].shape[0]), dtype=a.dtype, device=a.device)
                keep.append((s, a, saved))
            s, a = qp.qblock_norm(s, qp.qffn(a, *block, self.bits, self.gs, self.act, saved=saved), weight)
        if keep is not None:
            keep.append(s)
        return a

    def loss_and_gradients(self, ids, targets):
        """Of a model with norms: the mean loss, the gradients of weights() and of the norms."""
        keep, q = [], (self.bits, self.gs)
        a = self.normed(ids, keep)
        loss, lse = qp.qcross_entropy(a, targets, *self.head, *q)
        dloss = torch.full_like(loss, 1.0 / loss.numel())
        da, *head = qp.qcross_entropy_backward(a, targets, lse, dloss, *self.head, *q)
        s, ds, grads, norms = keep.pop(), None, [tuple(head)], []
        for block, weight in zip(reversed(self.blocks), reversed(self.norms)):
            before, a, saved = keep.pop()
            # The residual sum hands ds on to both its terms.
            ds, _, dw, _, _ = qp.qblock_norm_backward(s, da, ds, weight=weight)
            da, *pairs = qp.qffn_backward(a, ds, saved, *block, *q, self.act)
            grads, norms, s = [*pairs, *grads], [dw, *norms], before
        ds, _, dw, _, _ = qp.qblock_norm_backward(s, da, ds, weight=self.norms[0])
        table = qp.qembedding_backward(ids, ds, self.table[0], *q, self.factor)
        return loss.mean(), [table, *grads], [dw, *norms]


class Adam:
    """Adam over fp32 copies of the scales and biases; the model's own are rounded from them. A
    step is relative to the weight's first scales: a scale of 0.02 moves codes up to 255.
    (`norms`: more tensors, of their own first size.)"""

    def __init__(self, weights, lr, norms=()):
        self.t = 0
        self.lr = [lr * float(w[1].float().abs().mean()) for w in weights for _ in range(2)]
        self.lr += [lr * float(t.float().abs().mean()) for t in norms]
        self.params = [t for w in weights for t in w[1:]] + list(norms)
        self.master = [t.float() for t in self.params]
        self.m = [torch.zeros_like(t) for t in self.master]
        self.v = [torch.zeros_like(t) for t in self.master]

    def step(self, pairs, norms=()):
        self.t += 1
        grads = [g.float() for ds in pairs for g in ds] + [g.float() for g in norms]
        for p, w, m, v, g, lr in zip(self.params, self.master, self.m, self.v, grads, self.lr):
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.01)
            w -= lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8)
            p.copy_(w)


def train(model, steps, batch=256, lr=1e-2, seed=1, say=lambda s: None):
    """The mean loss of each step."""
    data = torch.tensor(list(TEXT.encode()), dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(seed)
    opt = Adam(model.weights(), lr, model.norms)
    losses = []
    for step in range(steps):
        at = torch.randint(0, data.numel() - 1, (batch,), generator=gen).cuda()
        ids, target = data[at], data[at + 1].long()
        if model.norms:
            loss, pairs, norms = model.loss_and_gradients(ids, data[at + 1])
            losses.append(loss)
            opt.step(pairs, norms)
        else:
            keep = []
            logits = model.forward(ids, keep).float()
            probs = torch.softmax(logits, 1)
            losses.append(torch.nn.functional.cross_entropy(logits, target))
            probs[torch.arange(batch, device="cuda"), target] -= 1
            opt.step(model.backward(ids, keep, (probs / batch).to(model.dtype)))
        if step % 20 == 0 or step == steps - 1:
            say(f"step {step}: loss {losses[-1].item():.3f}")
    return torch.stack(losses).tolist()


def allowed_bytes(chars):
    """A mask row of qlogits_adjust: one bit for each byte that may appear."""
    words = [0] * (VOCAB // 32)
    for c in set(chars.encode()):
        words[c // 32] |= 1 << (c % 32)
    words = [w - (1 << 32) if w >= 1 << 31 else w for w in words]
    return torch.tensor([words], dtype=torch.int32, device="cuda")


def decode(model, prompts, tokens, allowed, repetition=1.05, frequency=0.02, presence=0.0):
    """Greedy continuations of the prompts, all sequences a step."""
    rows = len(prompts)
    seqs = [list(p.encode()) for p in prompts]
    prompt_lens = torch.tensor([len(s) for s in seqs], dtype=torch.int32, device="cuda")
    rep, freq, pres = (torch.full((rows,), v, device="cuda") for v in (repetition, frequency, presence))
    mask = allowed_bytes(allowed)
    for _ in range(tokens):
        ids = torch.tensor([s[-1] for s in seqs], dtype=torch.int32, device="cuda")
        history = torch.tensor([t for s in seqs for t in s], dtype=torch.int32, device="cuda")
        ends = torch.tensor([0, *(len(s) for s in seqs)]).cumsum(0).to(torch.int32).cuda()
        logits = qp.qlogits_adjust(model.forward(ids), history, ends, prompt_lens, rep, freq, pres, mask=mask)
        for s, t in zip(seqs, logits.argmax(1).tolist()):
            s.append(t)
    return [bytes(s).decode(errors="replace") for s in seqs]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=4, choices=(2, 3, 4, 6, 8))
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--norms", action="store_true", help="norms between the blocks, and the loss without logits")
    a = ap.parse_args()
    model = TinyLM(bits=a.bits, seed=a.seed, norms=a.norms)
    train(model, a.steps, say=lambda s: print(s, flush=True))
    for line in decode(model, ["the c", "a rou", "step "], 24, "abcdefghijklmnopqrstuvwxyz .,"):
        print(repr(line))


if __name__ == "__main__":
    main()
