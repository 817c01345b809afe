"""A policy-gradient step of a small residual language model, out of this package's operators.

    x = dropout(embed(tokens))
    twice:  x = x + dropout(gated block(norm(x)))
    log probabilities and entropy of  norm(x) W_head^T

* every norm is ``pc_rmsnorm_store``: it drops out the last block's output, adds
  it to the residual, normalises, and stores what it gives in 8 bits on the way;
* what the backward pass needs is kept in 8 bits: each projection's input as the
  norm stored it, gate and up, and the residual sums;
* masks are kept nowhere: a seed and an offset, which live on the device and
  move on with each step, make them again in ``pc_rmsnorm_backward`` and
  ``pc_dropout``;
* the loss, ``- mean(advantage * logp) - beta * mean(entropy)``, goes through
  ``pc_logprobs`` and ``pc_logprobs_backward``, which writes the logits'
  gradient over the logits.

    python examples/residual_step.py [--steps N]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import static_codebook_lossless_amd as pc  # noqa: E402


class EmbedDropped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, mask):
        ctx.save_for_backward(tokens)
        ctx.rest = table.shape[0], table.dtype, scale, mask
        x = pc.pc_embed(tokens, table, scale=scale, dtype=torch.bfloat16)
        return pc.pc_dropout(x, mask, out=x)

    @staticmethod
    def backward(ctx, dx):
        (tokens,) = ctx.saved_tensors
        vocab, dtype, scale, mask = ctx.rest
        dx = pc.pc_dropout(dx.contiguous(), mask)
        return None, pc.pc_embed_backward(dx, tokens, vocab, scale=scale, dtype=dtype), None, None


class NormProject(torch.autograd.Function):
    """sum = residual + dropout(x);  (sum, norm(sum) W^T).  x None: the sum is the residual."""

    @staticmethod
    def forward(ctx, x, residual, gain, w, mask):
        if x is None:
            n = pc.pc_rmsnorm_store(residual, gain, y="plain")
        else:
            n = pc.pc_rmsnorm_store(x, gain, residual=residual, mask=mask, y="plain")
        ctx.save_for_backward(gain, w, n.rstd)
        ctx.kept = n.q, pc.pc_q8_store(n.sum)
        ctx.mask, ctx.alone = mask, x is None
        return (residual if x is None else n.sum), n.y @ w.to(n.y.dtype).t()

    @staticmethod
    def backward(ctx, d_sum, d_out):
        gain, w, rstd = ctx.saved_tensors
        q, total = ctx.kept
        d_out = d_out.contiguous()
        dw = pc.pc_q8_weight_grad(d_out, q, dtype=w.dtype)
        g = pc.pc_rmsnorm_backward(d_out @ w.to(d_out.dtype), total, gain, rstd,
                                   d_sum=None if d_sum is None else d_sum.contiguous(),
                                   mask=None if ctx.alone else ctx.mask, weight_dtype=gain.dtype)
        return None if ctx.alone else g.x, g.residual, g.weight, dw, None


class Gated(torch.autograd.Function):
    """(silu(gate) * up) W^T, gate and up side by side and kept in 8 bits."""

    @staticmethod
    def forward(ctx, gu, w):
        gate, up = gu.chunk(2, dim=1)
        ctx.save_for_backward(w)
        ctx.gu = pc.pc_q8_store(gu)
        return (torch.nn.functional.silu(gate) * up) @ w.to(gu.dtype).t()

    @staticmethod
    def backward(ctx, dy):
        (w,) = ctx.saved_tensors
        g = pc.pc_q8_glu_backward((dy @ w.to(dy.dtype)).contiguous(), ctx.gu, act="silu", with_h=True)
        return g.packed, (dy.t() @ g.h).to(w.dtype)


class LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens):
        r = pc.pc_logprobs(logits, tokens)
        ctx.save_for_backward(logits, tokens, r.stats)
        return r.logp, r.entropy

    @staticmethod
    def backward(ctx, d_logp, d_entropy):
        logits, tokens, stats = ctx.saved_tensors
        # nothing here reads the logits any more, so their gradient takes their place; a second backward
        # pass, or another loss that has saved them, gets autograd's error of a tensor modified in place
        return pc.pc_logprobs_backward(logits, stats, tokens, d_logp.contiguous(), d_entropy.contiguous(),
                                       out=logits.detach()), None


class Model:
    blocks = 2

    def __init__(self, vocab=512, dim=128, hidden=256, dropout=0.1, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-1])).requires_grad_()

        self.scale, self.dropout = math.sqrt(dim), dropout
        self.table, self.head = weight(vocab, dim), weight(vocab, dim)
        self.w_in = [weight(2 * hidden, dim) for _ in range(self.blocks)]
        self.w_out = [weight(dim, hidden) for _ in range(self.blocks)]
        self.gains = [torch.ones(dim, device=device).requires_grad_() for _ in range(self.blocks + 1)]
        self.random = torch.tensor([seed, 0], device=device)  # seed and step

    def parameters(self):
        return [self.table, self.head, *self.w_in, *self.w_out, *self.gains]

    def mask(self, layer):
        return pc.DropoutMask(self.dropout, self.random, offset=layer << 32)

    def logits(self, tokens):
        residual, x = EmbedDropped.apply(tokens, self.table, self.scale, self.mask(0)), None
        for k in range(self.blocks):
            residual, gu = NormProject.apply(x, residual, self.gains[k], self.w_in[k], self.mask(k))
            x = Gated.apply(gu, self.w_out[k])
        return NormProject.apply(x, residual, self.gains[-1], self.head, self.mask(self.blocks))[1]

    def loss(self, tokens, actions, advantage, beta=0.01):
        logp, entropy = LogProbs.apply(self.logits(tokens), actions)
        return -(advantage * logp).mean() - beta * entropy.mean()

    def next_step(self):
        self.random[1] += 1


def train(steps=8, tokens=1024, rate=0.5, report=print, **sizes):
    """Rewards one fixed successor of every token; returns each step's mean reward of sampled successors."""
    model = Model(**sizes)
    vocab, device = model.table.shape[0], model.table.device
    g = torch.Generator(device=device).manual_seed(1)
    successor = torch.randperm(vocab, generator=g, device=device)
    rewards = []
    for step in range(steps):
        t = torch.randint(0, vocab, (tokens,), generator=g, device=device)
        sampled = torch.randint(0, vocab, (tokens,), generator=g, device=device)
        actions = torch.where(torch.rand(tokens, generator=g, device=device) < 0.5, successor[t], sampled)
        reward = (actions == successor[t]).float()
        loss = model.loss(t, actions, reward - reward.mean())
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                p -= rate * p.grad
                p.grad = None
        model.next_step()
        rewards.append(float(reward.mean()))
        report("step %d: loss %.4f" % (step, float(loss.detach())))
    return rewards


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    train(steps=ap.parse_args().steps)
