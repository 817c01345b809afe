"""The example's training step: its gradients against plain ones in 64 bits, and that it trains."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture()
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_gradients(model, tokens, targets):
    """The same loss in 64 bits, through torch's own operators."""
    p = [q.detach().double().requires_grad_() for q in model.parameters()]
    table, w_in, w_out, head = p
    x = table[tokens] * model.scale
    gate, up = (x @ w_in.t()).chunk(2, dim=1)
    x = x + (torch.nn.functional.silu(gate) * up) @ w_out.t()
    torch.nn.functional.cross_entropy(x @ head.t(), targets).backward()
    return [q.grad for q in p]


def test_gradients(example):
    model = example.Model(vocab=300, dim=96, hidden=160, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for step in range(2):  # the second step's activations go through the coder
        tokens = torch.randint(0, 300, (700,), generator=g, device="cuda")
        targets = torch.randint(0, 300, (700,), generator=g, device="cuda")
        model.loss(tokens, targets).backward()
        for p, want in zip(model.parameters(), plain_gradients(model, tokens, targets)):
            # e4m3 keeps a number to a relative 2^-4, and bf16 adds a few 2^-8
            off = float((p.grad.double() - want).norm() / want.norm())
            assert off < 2.0 ** -4, off
            p.grad = None
    assert model.keep_gu.book is not None


def test_it_trains_in_fewer_bytes(example):
    losses, kept, plain = example.train(steps=10, tokens=4096, rate=4.0, report=lambda *_: None)
    assert losses[-1] < 0.9 * losses[0], losses
    assert kept < 0.53 * plain  # 8 bits and a 32nd of scales, less what the coder saves, plus its index
