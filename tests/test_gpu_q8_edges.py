"""Edges of the stored-tensor and embedding operators on the GPU: the ends of
their number ranges, against 64-bit forms.  Tolerances were fixed before the
first run and are derived where they are used.
"""
import math

import numpy as np
import pytest
import torch

from oracle import q8
from test_gpu_q8 import DEV, DT, _need_gpu, activation, make_q8, np64, rounded, same, tensor  # noqa: F401

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


# -- activation backward -------------------------------------------------------------

def test_gelu_keeps_its_digits_in_the_tail():
    # y = g P(g) of g below zero is all tail.  In steps of 2^-24 (half a unit
    # of 32 bits) its relative error is at most: b^2 / 2 times 2 of the
    # exponent's factor and its rounding, 2 of the exponential, 2 of the reciprocal times the
    # tail's slope in it (at most 8 over this range), 2 * 10 of ten
    # multiply-adds times their condition (below 2), 6 of the products around
    # them and the output's rounding
    g = -np.concatenate([np.arange(1, 128) / 128.0, np.arange(64, 128) / 64.0 * 2.0, np.arange(64, 128) / 64.0 * 4.0])
    rows = [np.pad(g[i:i + 32], (0, max(0, 32 - len(g[i:i + 32]))), mode="edge") for i in range(0, len(g), 32)]
    sym, codes = q8.store(np.array(rows), "int8")
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), "int8")
    v = q8.load(sym, codes, "int8")
    r = pc.pc_q8_glu_backward(torch.ones(v.shape, device=DEV), q, act="gelu", with_h=True)
    tail = np.vectorize(lambda x: 0.5 * math.erfc(x / math.sqrt(2.0)))(-v)
    want = v * tail
    tol = (v * v + 2 + 16 + 40 + 6) * 2.0 ** -24
    off = np.abs(np64(r.h) - want) / np.maximum(np.abs(want), 1e-300)
    assert np.all(np.where(want == 0, np64(r.h) == 0, off <= tol)), float((off / tol).max())
    # the slope is the difference of the tail and the density's product: the same, of either's size
    density = v * np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    assert np.all(np.abs(np64(r.gate) - (tail + density)) <= tol * (tail + np.abs(density)))


# -- embedding -----------------------------------------------------------------------

@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan, -2.0])
@pytest.mark.parametrize("table", ["f32", "bf16", "e4m3", "int8"])
def test_rows_outside_the_table_are_zero_for_every_scale(table, scale):
    rng = np.random.default_rng(35)
    tab = make_q8(rng, 9, 50, table)[0] if table in q8.MOST else activation(rng, 9, 50, table)
    tokens = torch.tensor([-1, 9, 1 << 35, 3], device=DEV)
    out = pc.pc_embed(tokens, tab, scale=scale, dtype=torch.float32)
    assert torch.all(out[:3] == 0)
    assert not torch.all(out[3] == 0)


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan, -2.0])
@pytest.mark.parametrize("n,vocab,dim", [(20, 300, 40), (300, 100, 33), (5000, 300, 40)])
def test_rows_without_a_token_are_zero_for_every_scale(n, vocab, dim, scale):
    rng = np.random.default_rng(36)
    tokens = rng.integers(0, vocab // 2, n)
    dy = activation(rng, n, dim, "f32")
    got = pc.pc_embed_backward(dy, torch.from_numpy(tokens).to(DEV), vocab, scale=scale)
    none = np.bincount(tokens, minlength=vocab) == 0
    assert torch.all(got[torch.from_numpy(none).to(DEV)] == 0)
    old = torch.full((vocab, dim), 4.0, device=DEV)
    pc.pc_embed_backward(dy, torch.from_numpy(tokens).to(DEV), vocab, scale=scale, out=old, accumulate=True)
    assert torch.all(old[torch.from_numpy(none).to(DEV)] == 4.0)


def test_embed_backward_of_many_tokens():
    # 2^28 tokens, a gradient of whole numbers that 32 bits hold
    g = torch.Generator(device=DEV).manual_seed(9)
    n, vocab = (1 << 28) + 5, 1000
    tokens = torch.randint(0, vocab, (n,), generator=g, device=DEV, dtype=torch.int32)
    dy = torch.randint(0, 4, (n,), generator=g, device=DEV, dtype=torch.int32)
    want = torch.zeros(vocab, dtype=torch.int64, device=DEV)
    for i in range(0, n, 1 << 26):
        both = torch.bincount(tokens[i:i + (1 << 26)] * 4 + dy[i:i + (1 << 26)], minlength=4 * vocab).view(vocab, 4)
        want += (both * torch.arange(4, device=DEV)).sum(1)
    got = pc.pc_embed_backward(dy.to(torch.bfloat16).view(n, 1), tokens, vocab)
    assert torch.equal(got.view(-1).long(), want)


def test_embed_backward_to_the_tallest_and_the_widest_table():
    dy = torch.tensor([[1.0], [2.0], [4.0], [8.0]], device=DEV)
    for vocab in ((1 << 26) - 5, (1 << 25) + 1):
        tokens = torch.tensor([vocab - 1, 0, vocab - 1, vocab // 2], device=DEV)
        got = pc.pc_embed_backward(dy, tokens, vocab)
        assert got[vocab - 1].item() == 5.0 and got[0].item() == 2.0 and got[vocab // 2].item() == 8.0
        assert torch.count_nonzero(got).item() == 3
        del got
    dim = 65537 * 512 - 3  # more slabs of columns than a launch has rows of workgroups
    wide = torch.ones(3, dim, device=DEV)
    wide[1, dim - 1] = 5.0
    got = pc.pc_embed_backward(wide, torch.tensor([1, 1, 3], device=DEV), 4)
    assert torch.all(got[0] == 0) and torch.all(got[2] == 0) and torch.all(got[3] == 1)
    assert torch.all(got[1, :-1] == 2) and got[1, -1].item() == 6.0


def test_weight_grad_of_no_rows_to_the_widest_result():
    k = (1 << 31) - 1024  # 2^24 - 8 tiles
    x = pc.Q8(torch.empty((0, k), dtype=torch.uint8, device=DEV), torch.empty((0, k // 32), dtype=torch.uint8, device=DEV))
    out = torch.full((1, k), 3.0, dtype=torch.bfloat16, device=DEV)
    none = torch.empty((0, 1), dtype=torch.float32, device=DEV)
    pc.pc_q8_weight_grad(none, x, dtype=torch.bfloat16, out=out, accumulate=True)
    assert torch.all(out == 3.0)
    pc.pc_q8_weight_grad(none, x, dtype=torch.bfloat16, out=out)
    assert torch.all(out == 0.0)


def test_the_binding_takes_numbers_and_refuses_others():
    table, tokens = torch.ones(5, 8, device=DEV), torch.tensor([1, 4], device=DEV)
    for scale in (2, 2.0, np.float32(2), torch.tensor(2.0)):
        assert torch.all(pc.pc_embed(tokens, table, scale=scale) == 2)
        assert pc.pc_embed_backward(table[:2], tokens, 5, scale=scale, padding=np.int64(4)).sum().item() == 16
    for call in (lambda: pc.pc_embed(tokens, table, scale="two"), lambda: pc.pc_embed(tokens, table, scale=None),
                 lambda: pc.pc_embed_backward(table[:2], tokens, 5, scale=[2]),
                 lambda: pc.pc_embed_backward(table[:2], tokens, 5, padding=0.5)):
        with pytest.raises((TypeError, ValueError)):
            call()
    q = pc.pc_q8_store(torch.randn(6, 70, device=DEV))
    wide = torch.zeros(6, 100, dtype=torch.uint8, device=DEV)
    wide[:, 5:75].copy_(q.symbols)
    for symbols in (q.symbols.reshape(-1), q.symbols.view(2, 3, 70), wide[:, 5:75], wide.view(2, 3, 100)[:, :, 5:75]):
        assert torch.equal(pc.pc_q8_load(q.with_symbols(symbols)), pc.pc_q8_load(q))
    for symbols in (q.symbols.reshape(-1)[:-1], q.symbols.t(), wide):
        with pytest.raises(ValueError):
            q.with_symbols(symbols)


# -- the ends of the range ------------------------------------------------------------

@pytest.mark.parametrize("fmt,limit", [("e4m3", 248 * 2.0 ** 120), ("int8", 127 * 2.0 ** 121)])
def test_the_top_of_the_range_rounds_to_infinity(fmt, limit):
    # magnitudes that round to 2^128 are stored as that, which 32 bits read as
    # infinity; below them everything is finite
    below = float(np.nextafter(np.float32(limit), np.float32(0)))
    most, most_bf16 = float(np.finfo(np.float32).max), 255 * 2.0 ** 120
    rows = [[v] + [1.0] * 31 for v in (below, most_bf16, -most_bf16, most, -most)]
    rows.append([most, below, -below, limit] + [0.0] * 28)
    x = np.array(rows, dtype=np.float32)
    q = pc.pc_q8_store(torch.from_numpy(x).to(DEV), fmt)
    sym, codes = q8.store(x.astype(np.float64), fmt)
    assert np.array_equal(q.symbols.cpu().numpy(), sym) and np.array_equal(q.scales.cpu().numpy(), codes)
    v = q8.load(sym, codes, fmt)
    assert np.array_equal(np.abs(v) == 2.0 ** 128, (np.abs(x) > limit) | ((x == limit) & (np.arange(32) == 3)))
    for to in ("f32", "bf16"):
        same(np64(pc.pc_q8_load(q, DT[to])), rounded(v, to))
    dy = np.zeros((6, 8), dtype=np.float32)
    dy[:, 0] = [1, 0, 0, 0, 0, 0]
    dy[:, 1] = [0, 1, 0, 0, 0, 0]
    with np.errstate(invalid="ignore"):
        want = dy.astype(np.float64).T @ rounded(v, "f32")
    for dtype in ("bf16", "f32"):
        same(np64(pc.pc_q8_weight_grad(tensor(dy, dtype), q)), rounded(want, "f32"))


def test_weight_grad_of_the_smallest_numbers():
    # the three terms of a 32-bit gradient are bf16 numbers, whose smallest
    # step is 2^-133: what lies below that is lost
    rng = np.random.default_rng(34)
    sym, codes = q8.store(rng.normal(size=(40, 64)) * 2.0 ** 60, "int8")
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), "int8")
    x = q8.load(sym, codes, "int8")
    for scale in (2.0 ** -100, 2.0 ** -112, 2.0 ** -122, 2.0 ** -130):
        dy = (rng.normal(size=(40, 24)) * scale).astype(np.float32)
        want, size = q8.weight_grad(dy.astype(np.float64), x), np.abs(dy.astype(np.float64)).T @ np.abs(x)
        lost = 2.0 ** -133 * np.abs(x).sum(axis=0)[None, :]
        off = np.abs(np64(pc.pc_q8_weight_grad(tensor(dy, "f32"), q)) - want)
        assert np.all(off <= 43 * 2.0 ** -23 * size + lost), (scale, float((off / size).max()))
