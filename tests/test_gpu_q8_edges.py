"""Edges of the stored-tensor and embedding operators on the GPU: the ends of
their number ranges, the sizes at which their launches change, and operands
past 4 GiB, against 64-bit forms.

Tolerances, fixed before the first run: as in test_gpu_q8.py, sums of m exact
terms in 32 bits are off by at most (m + 2) 2^-23 times the sum of the terms'
magnitudes, plus half a step of the output's type; others are derived where
they are used.
"""
import math

import numpy as np
import pytest
import torch

from oracle import q8
from test_gpu_q8 import (DEV, DT, HALF_STEP, TINY, _need_gpu, activation, check_glu, check_wgrad,  # noqa: F401
                         make_q8, np64, rounded, same, say, tensor)

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
    x = pc.Q8(torch.empty((0, k), dtype=torch.uint8, device=DEV),
              torch.empty((0, k // 32), dtype=torch.uint8, device=DEV))
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


# -- the sizes at which launches change, and operands past 4 GiB ----------------------

def test_glu_backward_of_stored_views():
    rng = np.random.default_rng(31)
    both, v = make_q8(rng, 6, 256, "int8", 2.0)
    dh = tensor(rng.normal(size=(6, 64)).astype(np.float32), "f32")
    gate, up = both.columns(32, 96), both.columns(160, 224)
    check_glu(np64(dh), v[:, 32:96], v[:, 160:224], "silu", "f32", pc.pc_q8_glu_backward(dh, gate, up))
    middle = both.columns(64, 192)  # gate and up side by side inside a wider tensor
    r = pc.pc_q8_glu_backward(dh, middle, with_h=True)
    check_glu(np64(dh), v[:, 64:128], v[:, 128:192], "silu", "f32", r, r.h)
    out = pc.pc_embed(torch.tensor([5, 0, 5], device=DEV), middle, dtype=torch.float32)
    same(np64(out), v[[5, 0, 5], 64:192])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,rows,cols", [("bf16", 2600, 2049), ("f32", 2600, 2049), ("bf16", 2600, 2048),
                                             ("f16", 20000, 250)])
def test_counted_store_in_several_rounds(dtype, rows, cols, fmt):
    # a counting workgroup takes 2048 units of 8 columns at a time, and 256 of
    # them 4 Mi elements a round: the last round here is a partial one
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(rows, cols, generator=g, device=DEV).mul_(3.0).to(DT[dtype])
    x[7, 3], x[rows - 1, cols - 1] = math.nan, math.inf
    counts = torch.full((256,), 5, dtype=torch.int64, device=DEV)
    q, plain = pc.pc_q8_store(x, fmt, counts=counts), pc.pc_q8_store(x, fmt)
    assert torch.equal(q.symbols, plain.symbols) and torch.equal(q.scales, plain.scales)
    assert torch.equal(counts - 5, torch.bincount(q.symbols.reshape(-1), minlength=256))
    for at in (slice(0, 9), slice(rows // 2, rows // 2 + 9), slice(rows - 9, rows)):
        sym, codes = q8.store(np64(x[at]), fmt)
        assert np.array_equal(q.symbols[at].cpu().numpy(), sym) and np.array_equal(q.scales[at].cpu().numpy(), codes)


@pytest.mark.parametrize("odt", ["f16", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight_grad_in_slices_to_16_bits(dtype, odt):
    rng = np.random.default_rng(32)
    q, x = make_q8(rng, 3001, 65, "e4m3", 0.1)
    dy = tensor(rng.normal(size=(3001, 31)).astype(np.float32) * 0.1, dtype)
    assert pc.pc_q8_weight_grad_workspace_bytes(3001, 31, 65) > 0
    check_wgrad(np64(dy), x, pc.pc_q8_weight_grad(dy, q, dtype=DT[odt]), odt)
    old = tensor(rng.normal(size=(31, 65)).astype(np.float32), odt)
    out = old.clone()
    pc.pc_q8_weight_grad(dy, q, dtype=DT[odt], out=out, accumulate=True)
    check_wgrad(np64(dy), x, out, odt, np64(old))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,k", [(100, 64), (104, 70)])
def test_weight_grad_of_operands_past_4_gib(n, k, fmt):
    # rows 32 MB and 16 MB apart: dy spans 10 GB, x 5 GB
    rng = np.random.default_rng(33)
    t, ld = 300, (1 << 24) - 8
    dy = torch.zeros((t - 1) * ld + n, dtype=torch.bfloat16, device=DEV).as_strided((t, n), (ld, 1))
    dy.copy_(activation(rng, t, n, "bf16"))
    sym, codes = q8.store(rng.normal(size=(t, k)), fmt)
    far = torch.zeros((t - 1) * ld + k, dtype=torch.uint8, device=DEV).as_strided((t, k), (ld, 1))
    far.copy_(torch.from_numpy(sym))
    q = pc.Q8(far, torch.from_numpy(codes).to(DEV), fmt)
    check_wgrad(np64(dy), q8.load(sym, codes, fmt), pc.pc_q8_weight_grad(dy, q), "f32")


def test_weight_grad_of_many_rows_past_4_gib():
    # 5 GB of dy without gaps, its rows shared among slices
    g = torch.Generator(device=DEV).manual_seed(6)
    t, n, k = 2_500_033, 1000, 48
    dy = torch.randn(t, n, generator=g, device=DEV, dtype=torch.bfloat16)
    q = pc.pc_q8_store(torch.randn(t, k, generator=g, device=DEV), "e4m3")
    got = pc.pc_q8_weight_grad(dy, q)
    want, size = torch.zeros(n, k, dtype=torch.float64, device=DEV), torch.zeros(n, k, dtype=torch.float64, device=DEV)
    for i in range(0, t, 1 << 18):
        a = dy[i:i + (1 << 18)].double().t().contiguous()
        b = pc.pc_q8_load(pc.Q8(q.symbols[i:i + (1 << 18)], q.scales[i:i + (1 << 18)]), torch.float32).double()
        want += torch.mm(a, b)
        size += torch.mm(a.abs_(), b.abs_())
    # no sum is longer than a slice's and its join
    assert bool((torch.abs(got.double() - want) <= (t + 3) * 2.0 ** -23 * size).all())
    assert float((got.double() - want).norm() / want.norm()) < 1e-4


def check_embed_backward(dy, tokens, vocab, odt="f32"):
    got = pc.pc_embed_backward(dy, tokens, vocab, dtype=DT[odt])
    dim = dy.shape[1]
    want = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV).index_add_(0, tokens, dy.double())
    size = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV).index_add_(0, tokens, dy.double().abs())
    terms = torch.bincount(tokens, minlength=vocab).unsqueeze(1)
    tol = (terms + 3) * 2.0 ** -23 * size
    assert bool((torch.abs(got.double() - want) <= tol + HALF_STEP[odt] * want.abs() + TINY[odt] * (size > 0)).all())
    assert torch.equal(got, pc.pc_embed_backward(dy, tokens, vocab, dtype=DT[odt]))
    old = torch.ones(vocab, dim, dtype=DT[odt], device=DEV)
    pc.pc_embed_backward(dy, tokens, vocab, dtype=DT[odt], out=old, accumulate=True)
    off = torch.abs(old.double() - (want + 1))
    assert bool((off <= tol + 2.0 ** -23 + HALF_STEP[odt] * (want + 1).abs()).all())
    assert bool((old[(terms == 0).view(-1)] == 1).all())


def some_tokens(g, n, vocab, skew):
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    if skew == "one":
        return torch.where(u < 0.9, torch.full_like(u, vocab // 2), u * vocab).long().clamp_(max=vocab - 1)
    return (u ** skew * vocab).long().clamp_(max=vocab - 1)


@pytest.mark.parametrize("skew", [1, 8, "one"])
@pytest.mark.parametrize("n", [511, 512, 513])
def test_embed_backward_at_the_change_of_launches(n, skew):
    # up to 512 tokens in one launch, of up to 16 rows of the table a workgroup; the last workgroup's range is short
    g = torch.Generator(device=DEV).manual_seed(7)
    for vocab, dim, dtype, odt in [(30001, 40, "bf16", "f32"), (15007, 601, "f32", "f32"), (34813, 512, "f16", "bf16"),
                                   (34816, 8, "f32", "f32"), (6553, 2051, "bf16", "f16")]:
        say("embed backward", n, vocab, dim, skew)
        dy = torch.randn(n, dim, generator=g, device=DEV).to(DT[dtype])
        check_embed_backward(dy, some_tokens(g, n, vocab, skew), vocab, odt)


@pytest.mark.parametrize("skew", [1, 8, "one"])
@pytest.mark.parametrize("dim", [2050, 2052])
def test_embed_backward_of_many_joins(dim, skew):
    # 1032 blocks of sorted tokens on 5 slabs of columns: 5155 ends of blocks that a run may cross
    g = torch.Generator(device=DEV).manual_seed(8)
    dy = torch.randn(33000, dim, generator=g, device=DEV).to(torch.bfloat16)
    check_embed_backward(dy, some_tokens(g, 33000, 3001, skew), 3001)


@pytest.mark.parametrize("dim", [7, 64, 1000])
def test_embed_backward_of_nothing_to_a_large_table(dim):
    none, no_tokens = torch.empty(0, dim, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    out = torch.full((100_003, dim), 2.0, device=DEV)
    pc.pc_embed_backward(none, no_tokens, 100_003, out=out, accumulate=True)
    assert torch.all(out == 2.0)
    pc.pc_embed_backward(none, no_tokens, 100_003, out=out)
    assert torch.all(out == 0.0)


@pytest.mark.parametrize("n,vocab", [(300, 500), (5000, 300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_backward_of_rows_that_end_where_memory_ends(dtype, n, vocab):
    # the last row's last column is the last of a 32 MiB allocation: nothing lies behind it
    g = torch.Generator(device=DEV).manual_seed(10)
    for dim in (4, 8, 33, 64, 252, 256, 260, 511, 516, 764, 1000):
        say("embed backward", n, dim, vocab, dtype)
        memory = torch.zeros((32 << 20) // DT[dtype].itemsize, dtype=DT[dtype], device=DEV)
        dy = memory[-n * dim:].view(n, dim)
        dy.copy_(torch.randn(n, dim, generator=g, device=DEV))
        tokens = some_tokens(g, n, vocab, 4)
        check_embed_backward(dy, tokens, vocab)
        old = torch.zeros((32 << 20) // 4, device=DEV)[-vocab * dim:].view(vocab, dim)
        pc.pc_embed_backward(dy, tokens, vocab, out=old, accumulate=True)
        assert torch.equal(old, pc.pc_embed_backward(dy, tokens, vocab))
        del memory, dy, old
