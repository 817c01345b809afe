"""Log probabilities where a lost or doubly counted element would show, and the order of their sums.

A row has one logit that counts: the others lie so far below that they add
nothing in 32 bits.  Then ln sum exp z is that logit, exactly but for one
rounding (its own exponential and the logarithm of 1, with what the rounded
reference lost: 8 u of it), and the entropy 0 (the same, and no more than 64 u
in all).  A lost element would leave a far lower number, one counted twice ln 2 more."""
import math

import numpy as np
import pytest
import torch

from test_gpu_step import DEV, DT, U, say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check_single(r, value, at, top):
    n = len(at)
    assert float((r.lse - value).abs().max()) <= 8 * U * value
    assert float(r.entropy.abs().max()) <= 64 * U
    assert float(r.logp.max()) <= 0 and float(r.logp.min()) >= -16 * U * value
    assert float((r.stats[:, 0] - value).abs().max()) == 0
    if top:
        assert torch.equal(r.top_index[:, 0], at) and r.top_index.shape == (n, top)


@pytest.mark.parametrize("low", [-1000.0, -math.inf])
@pytest.mark.parametrize("dtype,rows,vocab,top", [
    ("bf16", 4096, 1003, 0), ("f32", 600, 1003, 3), ("bf16", 300, 5003, 0), ("f16", 4097, 8190, 2),
    ("f32", 500, 17001, 0), ("f32", 600, 60001, 0), ("f32", 600, 60001, 5), ("bf16", 520, 98311, 0)])
def test_every_place_of_whole_rows(dtype, rows, vocab, top, low):
    say("single", dtype, rows, vocab, top, low)
    x = torch.full((rows, vocab), low, dtype=DT[dtype], device=DEV)
    lines = torch.arange(rows, device=DEV)
    for first in range(0, vocab, rows):
        at = (first + lines) % vocab
        x[lines, at] = 5.0
        check_single(pc.pc_logprobs(x, at, top=top), 5.0, at, top)
        x[lines, at] = low


@pytest.mark.parametrize("low", [-1000.0, -math.inf])
@pytest.mark.parametrize("dtype,rows,vocab,top", [
    ("bf16", 1, 131072, 0), ("bf16", 1, 131075, 4), ("f32", 3, 50257, 0), ("f16", 1, 700001, 1), ("f32", 256, 8195, 3),
    ("bf16", 40, 33001, 0)])
def test_places_of_split_rows(dtype, rows, vocab, top, low):
    say("single, split", dtype, rows, vocab, top, low)
    assert pc.pc_logprobs_workspace_bytes(rows, vocab, top, {"f32": 0, "f16": 1, "bf16": 2}[dtype]) > 0
    x = torch.full((rows, vocab), low, dtype=DT[dtype], device=DEV)
    lines = torch.arange(rows, device=DEV)
    # splits and lanes begin at multiples of 4 or 8 columns
    step = max(1, vocab * rows // 200000)
    places = [p for k in range(0, vocab, 512 * step) for p in (k, k + 3, k + 4, k + 7, k + 8, k + 511) if p < vocab]
    places += list(range(vocab - 40, vocab))
    for p in places:
        at = (p + 17 * lines) % vocab
        x[lines, at] = 5.0
        check_single(pc.pc_logprobs(x, at, top=top), 5.0, at, top)
        x[lines, at] = low


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 1, 5600000), ("bf16", 2, 2000000), ("f32", 1, 400001),
                                              ("f16", 5, 420000), ("f32", 7, 150000)])
def test_alternatives_change_no_sum(dtype, rows, vocab):
    """Sums of splits are added in one order, with alternatives or without."""
    g = torch.Generator(device=DEV).manual_seed(7)
    for k in range(12):
        say("order", dtype, rows, vocab, k)
        x = (torch.randn(rows, vocab, generator=g, device=DEV) * (0.5 + k)).to(DT[dtype])
        tokens = torch.randint(0, vocab, (rows, 3), generator=g, device=DEV)
        a, b = pc.pc_logprobs(x, tokens), pc.pc_logprobs(x, tokens, top=6)
        assert torch.equal(a.stats, b.stats) and torch.equal(a.logp, b.logp), k
