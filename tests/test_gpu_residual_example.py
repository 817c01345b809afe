"""The residual example's step: that it runs, and its gradients against plain ones in 64 bits with the same masks."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from oracle import step as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture()
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("residual_step", os.path.join(ROOT, "examples", "residual_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_gradients(model, tokens, actions, advantage, beta, seed, offset):
    p = [q.detach().double().requires_grad_() for q in model.parameters()]
    table, head = p[:2]
    w_in, w_out, gains = p[2:4], p[4:6], p[6:]
    n, dim = len(tokens), table.shape[1]

    def drop(x, layer):
        t = oracle.below(model.dropout)
        bits = torch.from_numpy(oracle.numbers(n, dim, seed, (layer << 32) + offset).astype("int64")).to(x.device)
        return torch.where(bits < t, torch.zeros_like(x), x * (65536 / (65536 - t)))

    def norm(x, gain):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * gain

    x = drop(table[tokens] * model.scale, 0)
    for k in range(2):
        gate, up = (norm(x, gains[k]) @ w_in[k].t()).chunk(2, dim=1)
        x = x + drop((gate * torch.sigmoid(gate) * up) @ w_out[k].t(), k + 1)
    logp = torch.log_softmax(norm(x, gains[2]) @ head.t(), 1)
    entropy = -(logp.exp() * logp).sum(1)
    picked = logp.gather(1, actions[:, None])[:, 0]
    (-(advantage.double() * picked).mean() - beta * entropy.mean()).backward()
    return [q.grad for q in p]


def test_gradients(example):
    model = example.Model(vocab=300, dim=96, hidden=160, dropout=0.2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for k in range(2):
        tokens = torch.randint(0, 300, (700,), generator=g, device="cuda")
        actions = torch.randint(0, 300, (700,), generator=g, device="cuda")
        advantage = torch.randn(700, generator=g, device="cuda")
        model.loss(tokens, actions, advantage, beta=0.3).backward()
        want = plain_gradients(model, tokens, actions, advantage, 0.3, 3, k)
        for p, w in zip(model.parameters(), want):
            # e4m3 keeps a number to a relative 2^-4, and each of the two blocks' backward passes uses such ones;
            # bf16 adds a few 2^-8
            off = float((p.grad.double() - w).norm() / w.norm())
            assert off < 2.0 ** -3, (tuple(p.shape), off)
            p.grad = None
        model.next_step()


def test_it_runs(example):
    rewards = example.train(steps=3, tokens=512, report=lambda *_: None)
    assert len(rewards) == 3


def test_steps_draw_new_masks(example):
    model = example.Model(dropout=0.5)
    tokens = torch.arange(64, device="cuda")
    first = model.logits(tokens).detach()
    assert torch.equal(first, model.logits(tokens).detach())
    model.next_step()
    assert not torch.equal(first, model.logits(tokens).detach())
