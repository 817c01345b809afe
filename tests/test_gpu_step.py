"""The norm, dropout and log-probability operators on the GPU against their
plain 64-bit forms (oracle/step.py).

Tolerances, fixed before the first run; u = 2^-24, and half a step of an
output's type (a relative 2^-24, 2^-11 or 2^-8) and its smallest number come on
top everywhere:
* dropout: one product in 32 bits, rounded to the type: equal.
* norm: the sum has 3 u of each addend.  Everything else is compared with what
  follows from the sum as it was written: rstd comes from 64 bits with one
  rounding (1.01 u), y has two products more (3.1 u).  The stored form is that
  of y in 64 bits, byte for byte: both sides are within 2^-44 of y before the
  one rounding, so a difference has a chance of one in 10^7 for a million elements.
* norm's backward pass: a sum of a row's terms passes through at most
  D = 64 + cols / 1024 additions for any one term (8 or 16 in a lane's units,
  one more each for every 1024 x 8 columns, 6 over the lanes, 16 over the waves),
  each off by u of what is summed, so mean(g n) by (D + 4) u mean|g n|.  The
  weight's gradient adds rows one after the other: (rows + 40) u of the terms'
  magnitudes.
* log probabilities: with y = scale (x - max), an exponential's argument is off
  by 4 u |y| and the exponential by 2 u more; weighted by the probabilities the
  mean |y| is entropy - ln S <= entropy; a term passes through at most
  vocab / 64 + 64 additions.  So ln S is off by
  d = (vocab / 64 + 70 + 4 entropy) u + 2 u |ln S|, a log probability by
  d + 4 u (|y| + |logp|), the entropy by (3 d + 20 u)(1 + entropy + |ln S|).
  A probability's relative error is that of its logarithm plus 4 u |logp| + 2 u.
"""
import sys

import numpy as np
import pytest
import torch

from oracle import q8, step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}
U = 2.0 ** -24
EPS = float(np.float32(1e-6))


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.detach().double().cpu().numpy()


def tensor(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype]).to(DEV)


def activation(rng, rows, cols, dtype, size=1.0):
    return tensor((rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1))) * size).astype(np.float32), dtype)


def within(got, want, tol, dtype="f32"):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape
    off = np.abs(got - want) - (tol + HALF_STEP[dtype] * np.abs(want) + TINY[dtype])
    assert np.all(np.isfinite(got)) and np.all(off <= 0), (float(off.max()), int((off > 0).sum()))


def same(got, want):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape
    ok = (got == want) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (int((~ok).sum()), got[~ok][:4], want[~ok][:4])


# -- dropout -------------------------------------------------------------------

MASK_SIZES = [(1, 1), (1, 7), (3, 8), (5, 33), (2, 1000), (130, 96), (7, 4099), (1029, 16)]


def dropped(x, p, seed, offset):
    """mask(x) as 32 bits give it, x a tensor."""
    t = step.below(p)
    gone = torch.from_numpy(step.numbers(*x.shape, seed, offset) < t).to(x.device)
    keep = np.float32(65536 / (65536 - t)) if t < 65536 else np.float32(0)
    return torch.where(gone, torch.zeros((), device=x.device), x.float() * float(keep)).to(x.dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(dtype, p):
    rng = np.random.default_rng(11)
    for rows, cols in MASK_SIZES:
        say("dropout", rows, cols, dtype, p)
        x = activation(rng, rows, cols, dtype)
        seed, offset = int(rng.integers(1 << 63)) * 2 + 1, int(rng.integers(1 << 63)) * 2
        want = dropped(x, p, seed, offset)
        got = pc.pc_dropout(x, pc.DropoutMask(p, seed, offset))
        assert got.dtype == x.dtype and torch.equal(got, want)
        # seed and offset on the device, the offset in two parts
        where = torch.tensor([seed - (1 << 64) if seed >> 63 else seed, 12345], device=DEV)
        got = pc.pc_dropout(x, pc.DropoutMask(p, where, (offset - 12345) % (1 << 64)))
        assert torch.equal(got, want)
        got = pc.pc_dropout(x, pc.DropoutMask(p, seed, offset), out=x)  # in place
        assert got is x and torch.equal(x, want)


def test_dropout_rows_keep_their_masks():
    """The mask goes by row and column: strides, more rows and more columns change nothing."""
    rng = np.random.default_rng(12)
    x = activation(rng, 40, 200, "bf16")
    mask = pc.DropoutMask(0.3, 5, 6)
    whole = pc.pc_dropout(x, mask)
    assert torch.equal(pc.pc_dropout(x[:17, :75], mask), whole[:17, :75])
    assert torch.equal(pc.pc_dropout(x.view(4, 10, 200), mask).view(40, 200), whole)
    out = torch.full((40, 300), 7.0, dtype=torch.bfloat16, device=DEV)
    pc.pc_dropout(x[:, :199], mask, out=out[:, 3:202])
    assert torch.equal(out[:, 3:202], whole[:, :199])
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 202:] == 7).all())
    assert pc.pc_dropout(x[0], mask).shape == (200,)
    for seed, offset in ((6, 6), (5, 7), (5, 6 + (1 << 32)), (5 + (1 << 32), 6)):
        assert not torch.equal(pc.pc_dropout(x, pc.DropoutMask(0.3, seed, offset)), whole)


# -- norm ----------------------------------------------------------------------

NORM_SIZES = [(1, 1), (2, 7), (3, 31), (5, 32), (4, 33), (9, 100), (3, 511), (2, 513), (5, 1000), (515, 520), (3, 2048),
              (2, 2056), (600, 1032), (2, 4097), (514, 4100), (1, 8192), (3, 8200), (516, 8200), (2, 16392), (2, 32776),
              (1, 40001)]


def check_stored(q, y, fmt):
    sym, codes = q8.store(y, fmt)
    assert np.array_equal(q.scales.cpu().numpy(), codes)
    assert np.array_equal(q.symbols.cpu().numpy(), sym)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"),
                                       ("bf16", None)])
def test_rmsnorm_store(dtype, res, fmt):
    rng = np.random.default_rng(13)
    for k, (rows, cols) in enumerate(NORM_SIZES):
        say("norm", rows, cols, dtype, res, fmt)
        x = activation(rng, rows, cols, dtype)
        residual = None if res is None else activation(rng, rows, cols, res, 3.0)
        w_kind = ["f32", dtype, "bf16", None][k % 4]
        weight = None if w_kind is None else tensor((1 + 0.3 * rng.normal(size=cols)).astype(np.float32), w_kind)
        p, seed, offset = [0.0, 0.25][k % 2], 1234567 + k, 1 << 40
        mask = pc.DropoutMask(p, seed, offset) if p else None
        counts = torch.full((256,), 2, dtype=torch.int64, device=DEV)
        r = pc.pc_rmsnorm_store(x, weight, residual, mask, eps=1e-6, format=fmt, counts=counts, y="plain")
        # the sum
        total = step.dropout(np64(x), p, seed, offset)
        size = np.abs(total)
        if residual is not None:
            total, size = total + np64(residual), size + np.abs(np64(residual))
        sum_type = res or dtype
        if residual is None and mask is None:
            assert r.sum is x
        else:
            assert r.sum.dtype == DT[sum_type]
            within(np64(r.sum), total, 3 * U * size, sum_type)
        # what follows from it
        h = np64(r.sum)
        y, rstd = step.norm(h, np64(weight) if weight is not None else 1.0, EPS)
        off = np.abs(np64(r.rstd) - rstd) / rstd
        assert off.max() <= 1.01 * U, off.max()
        within(np64(r.y), y, 3.1 * U * np.abs(y), dtype)
        check_stored(r.q, y, fmt)
        symbols = r.q.symbols.cpu().numpy()
        assert np.array_equal(counts.cpu().numpy(), 2 + np.bincount(symbols.reshape(-1), minlength=256))
        # the other forms of the call give the same
        s = pc.pc_rmsnorm_store(x, weight, residual, mask, eps=1e-6, format=fmt, y="stored", dtype=torch.bfloat16)
        assert torch.equal(s.q.symbols, r.q.symbols) and torch.equal(s.q.scales, r.q.scales)
        assert torch.equal(s.y, pc.pc_q8_load(r.q, torch.bfloat16))
        assert torch.equal(s.rstd, r.rstd) and torch.equal(s.sum, r.sum)
        s = pc.pc_rmsnorm_store(x, weight, residual, mask, eps=1e-6, format=None, y="plain", dtype=torch.float32)
        assert s.q is None and torch.equal(s.y.to(DT[dtype]), r.y) and torch.equal(s.sum, r.sum)
        if residual is not None:
            s = pc.pc_rmsnorm_store(x, weight, residual, mask, eps=1e-6, format=fmt, sum_out=residual)  # in place
            assert s.sum is residual and torch.equal(residual, r.sum)
            assert torch.equal(s.q.symbols, r.q.symbols) and s.y is None


@pytest.mark.parametrize("kept", ["plain", "e4m3", "int8"])
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
def test_rmsnorm_backward(dtype, res, kept):
    rng = np.random.default_rng(14)
    for k, (rows, cols) in enumerate(NORM_SIZES):
        say("norm backward", rows, cols, dtype, res, kept)
        dy = activation(rng, rows, cols, dtype)
        total = activation(rng, rows, cols, res, 3.0)
        h = np64(total)
        if kept != "plain":
            sym, codes = q8.store(h, kept)
            total = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), kept)
            h = q8.load(sym, codes, kept)
        rstd = tensor(step.rstd(h, EPS).astype(np.float32), "f32")
        w_kind = ["f32", dtype, "bf16", None][k % 4]
        weight = None if w_kind is None else tensor((1 + 0.3 * rng.normal(size=cols)).astype(np.float32), w_kind)
        d_sum = activation(rng, rows, cols, res) if k % 3 else None
        p, seed, offset = [0.0, 0.25][k % 2], 77 + k, k << 33
        mask = pc.DropoutMask(p, seed, offset) if p else None
        r = pc.pc_rmsnorm_backward(dy, total, weight, rstd, d_sum=d_sum, mask=mask, dtype=DT[res])
        w64 = np64(weight) if weight is not None else np.ones(cols)
        ds = np64(d_sum) if d_sum is not None else np.zeros((rows, cols))
        d, dw = step.norm_backward(np64(dy), h, w64, np64(rstd), ds)
        n, r64 = h * np64(rstd)[:, None], np64(rstd)[:, None]
        g = np64(dy) * w64
        depth = 64 + cols / 1024
        tol = U * (r64 * (6 * np.abs(g) + (depth + 8) * np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
                   + 2 * np.abs(ds) + 2 * np.abs(d))
        assert r.residual.dtype == DT[res]
        within(np64(r.residual), d, tol, res)
        if p == 0 and res == dtype:
            assert r.x is r.residual
        else:
            keep = 65536 / (65536 - step.below(p))
            assert r.x.dtype == DT[dtype]
            within(np64(r.x), step.dropout(d, p, seed, offset), keep * (tol + 3 * U * np.abs(d)), dtype)
        if weight is None:
            assert r.weight is None
            continue
        dw_tol = (rows + 40) * U * np.abs(np64(dy) * n).sum(0)
        within(np64(r.weight), dw, dw_tol)
        # into a given tensor of another type, and added to one
        for kind in ("f32", "bf16"):
            old = tensor(rng.normal(size=cols).astype(np.float32), kind)
            before = np64(old)
            s = pc.pc_rmsnorm_backward(dy, total, weight, rstd, d_sum=d_sum, mask=mask, dtype=DT[res],
                                       weight_dtype=DT[kind], weight_out=old, accumulate=True)
            assert s.weight is old and torch.equal(s.residual, r.residual) and torch.equal(s.x, r.x)
            within(np64(old), before + dw, dw_tol + U * np.abs(before + dw), kind)


# -- log probabilities -----------------------------------------------------------

LOGIT_SIZES = [(1, 1, 1, 1), (3, 5, 2, 5), (2, 64, 1, 64), (5, 100, 64, 7), (4, 1000, 3, 50), (7, 2049, 1, 20),
               (1, 4099, 2, 64), (2, 8193, 1, 1), (600, 777, 1, 3), (515, 5003, 2, 10), (1, 50257, 1, 20),
               (3, 128000, 5, 50), (40, 20011, 1, 0)]


def logits(rng, rows, vocab, dtype):
    x = rng.normal(size=(rows, vocab)) * 3
    liked = rng.integers(0, vocab, size=rows)
    x[np.arange(rows), liked] += 8
    return tensor(x.astype(np.float32), dtype), liked


def spread(x64, scale, entropy, vocab):
    """(y, ln S, the bound of ln S's error)"""
    y = (x64 - x64.max(1, keepdims=True)) * scale
    log_s = np.log(np.exp(y).sum(1))
    return y, log_s, U * (vocab / 64 + 70 + 4 * entropy) + 2 * U * np.abs(log_s)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.6, 1.7])
def test_logprobs(dtype, scale):
    rng = np.random.default_rng(15)
    s64 = float(np.float32(scale))
    for rows, vocab, m, top in LOGIT_SIZES:
        say("logprobs", rows, vocab, m, top, dtype, scale)
        x, liked = logits(rng, rows, vocab, dtype)
        tokens = rng.integers(0, vocab, size=(rows, m))
        tokens[:, 0] = liked
        t = torch.from_numpy(tokens).to(DEV)
        r = pc.pc_logprobs(x, t if m > 1 else t[:, 0], top=top, scale=scale)
        x64 = np64(x)
        logp, entropy, index, top_logp = step.logprobs(x64, tokens, s64, top)
        y, log_s, d = spread(x64, s64, entropy, vocab)
        got = np64(r.logp).reshape(rows, m)
        at = np.take_along_axis(y, tokens, 1)
        within(got, logp, d[:, None] + 4 * U * (np.abs(at) + np.abs(logp)))
        within(np64(r.entropy), entropy, (3 * d + 20 * U) * (1 + entropy + np.abs(log_s)))
        lse = x64.max(1) * s64 + log_s
        within(np64(r.lse), lse, d + 3 * U * (np.abs(lse) + np.abs(log_s)))
        if top:
            assert np.array_equal(r.top_index.cpu().numpy(), index)
            at = np.take_along_axis(y, index, 1)
            within(np64(r.top_logp), top_logp, d[:, None] + 4 * U * (np.abs(at) + np.abs(top_logp)))
        else:
            assert r.top_index is None and r.top_logp is None
        again = pc.pc_logprobs(x, t.to(torch.int32) if m > 1 else t[:, 0].to(torch.int32), scale=scale)
        assert torch.equal(again.logp, r.logp) and torch.equal(again.stats, r.stats)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("with_entropy", [False, True])
def test_logprobs_backward(dtype, with_entropy):
    rng = np.random.default_rng(16)
    for k, (rows, vocab, m, _) in enumerate(LOGIT_SIZES):
        say("logprobs backward", rows, vocab, m, dtype, with_entropy)
        scale = [1.0, 0.7][k % 2]
        s64 = float(np.float32(scale))
        x, liked = logits(rng, rows, vocab, dtype)
        tokens = rng.integers(0, vocab, size=(rows, m))
        tokens[:, 0] = liked
        if m > 2:
            tokens[:, 2] = tokens[:, 1]  # the same token twice
        tokens[::5, m - 1] = -1
        d_logp = rng.normal(size=(rows, m)).astype(np.float32)
        d_entropy = rng.normal(size=rows).astype(np.float32)
        t = torch.from_numpy(tokens).to(DEV)
        shape = (rows, m) if m > 1 else (rows,)
        r = pc.pc_logprobs(x, t.view(shape), scale=scale)
        args = (r.stats, t.view(shape), torch.from_numpy(d_logp).to(DEV).view(shape))
        more = dict(scale=scale, d_entropy=torch.from_numpy(d_entropy).to(DEV) if with_entropy else None)
        got = pc.pc_logprobs_backward(x, *args, **more)
        assert got.dtype == x.dtype
        x64 = np64(x)
        de = d_entropy.astype(np.float64) if with_entropy else np.zeros(rows)
        want = step.logprobs_backward(x64, tokens, s64, d_logp.astype(np.float64), de)
        logp = step.log_softmax(x64, s64)
        p = np.exp(logp)
        entropy = -(p * logp).sum(1)
        y, log_s, d = spread(x64, s64, entropy, vocab)
        rel = d[:, None] + 4 * U * (np.abs(y) + np.abs(logp)) + 4 * U * np.abs(logp) + 2 * U  # of p
        used = np.where(tokens >= 0, np.abs(d_logp), 0.0).sum(1, keepdims=True)
        off_entropy = ((3 * d + 20 * U) * (1 + entropy + np.abs(log_s)))[:, None]
        size = used + np.abs(de)[:, None] * (np.abs(logp) + entropy[:, None])
        given = np.zeros((rows, vocab))  # what the tokens add, where they add
        for row, at, g in zip(given, tokens, d_logp):
            np.add.at(row, at[at >= 0], np.abs(g[at >= 0]))
        tol = s64 * (p * size * (rel + (m + 12) * U) + p * np.abs(de)[:, None] * (off_entropy + rel)
                     + (m + 4) * U * (given + (given > 0) * p * size))
        within(np64(got), want, tol, dtype)
        assert torch.equal(pc.pc_logprobs_backward(x, *args, out=x, **more), got)  # in place
        assert torch.equal(x, got)
