"""A training step whose activations are kept in 8 bits and entropy coded.

A small language model -- an embedding, one gated feed-forward block and an
output projection -- trained on synthetic tokens:

* the embedding is ``pc_embed``, its gradient ``pc_embed_backward``;
* the block keeps its input and its gate and up projections with
  ``pc_q8_store``, counted on the way;
* the counts go to a ``CodebookRefresh`` per tensor, whose codebook, built
  from earlier steps, codes the next step's symbols with ``pc_encode``;
* the backward pass gets them back with ``pc_decode`` and uses them as they
  are: ``pc_q8_glu_backward`` and ``pc_q8_weight_grad``.

    python examples/train_step.py [--steps N]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import static_codebook_lossless_amd as pc  # noqa: E402

CHUNK = 16384


class Keeper:
    """Stores one tensor of every step: 8 bits, then the codebook of earlier steps."""

    def __init__(self, fmt="e4m3"):
        self.format = fmt
        self.refresh = pc.CodebookRefresh("huffman", window=4)
        self.book = None          # the codebook on the device
        self.bytes = self.plain_bytes = 0

    def keep(self, x):
        counts = torch.zeros(256, dtype=torch.int64, device=x.device)
        q = pc.pc_q8_store(x, self.format, counts=counts)
        self.plain_bytes = x.numel() * x.element_size()
        kept = q
        if self.book is not None:
            enc = pc.pc_encode(self.book, q.symbols, CHUNK)
            words = int(enc.chunk_word_offset[-1].item())
            if int(enc.status.item()) != pc.PC_OK:
                raise pc.PcError(int(enc.status.item()), "pc_encode")
            # the full-capacity payload buffer is given back, and the symbols with it
            enc = enc._replace(payload=enc.payload[:max(words, 4)].clone())
            self.bytes = sum(t.numel() * t.element_size() for t in
                             (enc.payload, enc.chunk_bits, enc.chunk_word_offset, enc.sub_off, q.scales))
            kept = (self.book, enc, q.symbols.shape, q.scales)
        else:
            self.bytes = q.symbols.numel() + q.scales.numel()
        if self.refresh.observe(counts):
            self.book = self.refresh.codebook.to(x.device)
        return kept

    def get(self, kept) -> pc.Q8:
        if isinstance(kept, pc.Q8):
            return kept
        book, enc, shape, scales = kept
        symbols, status = pc.pc_decode(book, enc)
        if int(status.item()) != pc.PC_OK:
            raise pc.PcError(int(status.item()), "pc_decode")
        return pc.Q8(symbols.view(shape), scales, self.format)


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale):
        ctx.save_for_backward(tokens)
        ctx.table, ctx.scale = (table.shape[0], table.dtype), scale
        return pc.pc_embed(tokens, table, scale=scale, dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, dy):
        (tokens,) = ctx.saved_tensors
        vocab, dtype = ctx.table
        return None, pc.pc_embed_backward(dy.contiguous(), tokens, vocab, scale=ctx.scale, dtype=dtype), None


class GatedBlock(torch.autograd.Function):
    """y = (silu(x Wg^T) * (x Wu^T)) Wd^T, W_gate and W_up in one [2 f, d] matrix."""

    @staticmethod
    def forward(ctx, x, w_in, w_out, keep_x, keep_gu):
        gu = x @ w_in.to(x.dtype).t()
        gate, up = gu.chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ w_out.to(x.dtype).t()
        ctx.save_for_backward(w_in, w_out)
        ctx.x, ctx.gu = keep_x.keep(x), keep_gu.keep(gu)
        ctx.keepers = keep_x, keep_gu
        return y

    @staticmethod
    def backward(ctx, dy):
        w_in, w_out = ctx.saved_tensors
        keep_x, keep_gu = ctx.keepers
        dy = dy.contiguous()
        dh = dy @ w_out.to(dy.dtype)
        g = pc.pc_q8_glu_backward(dh, keep_gu.get(ctx.gu), act="silu", with_h=True)
        d_in = pc.pc_q8_weight_grad(g.packed, keep_x.get(ctx.x), dtype=w_in.dtype)
        d_out = (dy.t() @ g.h).to(w_out.dtype)
        return g.packed @ w_in.to(dy.dtype), d_in, d_out, None, None


class Model:
    def __init__(self, vocab=512, dim=128, hidden=256, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, size):
            return (torch.randn(*shape, generator=g, device=device) * size).requires_grad_()

        self.scale = math.sqrt(dim)
        self.table = weight(vocab, dim, size=1 / math.sqrt(dim))
        self.w_in = weight(2 * hidden, dim, size=1 / math.sqrt(dim))
        self.w_out = weight(dim, hidden, size=1 / math.sqrt(hidden))
        self.head = weight(vocab, dim, size=1 / math.sqrt(dim))
        self.keep_x, self.keep_gu = Keeper(), Keeper()

    def parameters(self):
        return [self.table, self.w_in, self.w_out, self.head]

    def loss(self, tokens, targets):
        x = Embed.apply(tokens, self.table, self.scale)
        x = x + GatedBlock.apply(x, self.w_in, self.w_out, self.keep_x, self.keep_gu)
        return torch.nn.functional.cross_entropy(x.float() @ self.head.t(), targets)


def train(steps=8, tokens=1024, rate=0.5, report=print, **sizes):
    """Trains on a fixed successor for every token; returns the losses and the last step's kept and plain bytes."""
    model = Model(**sizes)
    vocab, device = model.table.shape[0], model.table.device
    g = torch.Generator(device=device).manual_seed(1)
    successor = torch.randperm(vocab, generator=g, device=device)
    losses = []
    for step in range(steps):
        t = torch.randint(0, vocab, (tokens,), generator=g, device=device)
        loss = model.loss(t, successor[t])
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                p -= rate * p.grad
                p.grad = None
        losses.append(float(loss.detach()))
        kept = model.keep_x.bytes + model.keep_gu.bytes
        plain = model.keep_x.plain_bytes + model.keep_gu.plain_bytes
        report("step %d: loss %.4f, activations kept in %d bytes (%.1f%% of bf16)"
               % (step, losses[-1], kept, 100.0 * kept / plain))
    return losses, kept, plain


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    train(steps=ap.parse_args().steps)
