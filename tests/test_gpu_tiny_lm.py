"""examples/tiny_lm.py: the operators together. Training on scales and biases
lowers the loss of a predictable text, the same seed gives the same losses,
and decoding keeps to the mask."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from qhelpers import log

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tiny_lm.py")


def example():
    spec = importlib.util.spec_from_file_location("tiny_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits,gs,act,dtype", [
    (4, 32, "silu", torch.bfloat16), (8, 64, "gelu_tanh", torch.float32), (3, 128, "silu", torch.float16)])
def test_training_lowers_the_loss_and_decoding_keeps_to_the_mask(bits, gs, act, dtype):
    lm = example()
    runs = []
    for _ in range(2):
        log(f"tiny model: {bits} bits, groups of {gs}, {act}, {dtype}")
        model = lm.TinyLM(bits=bits, group_size=gs, act=act, dtype=dtype)
        losses = lm.train(model, 80)
        out = lm.decode(model, ["the", "a tok"], 12, "abcdefghijklmnopqrstuvwxyz .")
        runs.append((losses, out))
    assert runs[0] == runs[1]
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert last < 0.6 * first, (first, last)
    for prompt, text in zip(["the", "a tok"], out):
        assert text.startswith(prompt) and len(text) == len(prompt) + 12
        assert set(text) <= set("abcdefghijklmnopqrstuvwxyz .")
