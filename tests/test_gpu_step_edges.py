"""The norm, dropout and log-probability operators at the ends of the number
ranges, at masks that leave little or nothing, with strides, shapes and streams
other than the plain ones, in captured graphs, past 4 GiB, and where launches
change.  Tolerances are those of test_gpu_step.py."""
import math

import numpy as np
import pytest
import torch

from oracle import q8, step
from test_gpu_step import (DEV, DT, EPS, HALF_STEP, U, activation, check_stored, dropped, logits, np64, same, say, spread,
                           tensor, within)

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc

INF, NAN = math.inf, math.nan
LOWEST = {k: float(torch.finfo(v).min) for k, v in DT.items()}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# -- dropout -------------------------------------------------------------------

def test_dropped_elements_are_zero_whatever_they_held():
    x = torch.full((64, 256), NAN, device=DEV)
    x[::2] = INF
    y = pc.pc_dropout(x, pc.DropoutMask(0.5, 1))
    gone = torch.from_numpy(step.numbers(64, 256, 1, 0) < 32768).to(DEV)
    assert bool((y[gone] == 0).all()) and not bool(torch.isfinite(y[~gone]).any())
    assert not bool(pc.pc_dropout(x, pc.DropoutMask(1.0, 1)).any())


def test_small_and_large_shares():
    x = torch.ones(512, 512, device=DEV)
    assert torch.equal(pc.pc_dropout(x, pc.DropoutMask(2.0 ** -18, 1)), x)  # nearer to none than to one in 65536
    for t in (1, 65535):
        y = pc.pc_dropout(x, pc.DropoutMask(t / 65536, 9, 8))
        want = step.numbers(512, 512, 9, 8) >= t
        assert np.array_equal(y.cpu().numpy() != 0, want)
        assert float(y.max()) in (0.0, float(np.float32(65536 / (65536 - t))))


def test_dropout_of_rows_past_4_gib():
    rows, cols = 70001, 33000  # 4.3 GiB of bf16
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    mask = pc.DropoutMask(0.5, 77, 88)
    y = pc.pc_dropout(x, mask, out=x)
    for r in (0, 1, 32537, 65075, 65076, rows - 1):  # 2^31 elements are passed in row 65075
        bits = numbers_of_row(r, cols, 77, 88)
        assert np.array_equal(y[r].float().cpu().numpy() == 0, bits < 32768), r


def numbers_of_row(row, cols, seed, offset):
    out = []
    for b in range(-(-cols // 8)):
        for w in step.philox((b, row, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32)):
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:cols])


# -- norm ------------------------------------------------------------------------

def test_norm_of_padding_and_extremes():
    """Rows of zeros, of the largest and smallest numbers, and with infinities and NaN."""
    cols = 200
    x = np.zeros((8, cols), dtype=np.float32)
    x[1] = 3e38
    x[2] = -1e-30
    x[3, 5] = INF
    x[4, 6] = NAN
    x[5] = np.linspace(-1, 1, cols)
    x[6] = 1e-45
    x[7, ::2] = 2e19
    t = torch.from_numpy(x).to(DEV)
    r = pc.pc_rmsnorm_store(t, eps=1e-6, y="plain")
    assert r.sum is t
    y, rstd = step.norm(x.astype(np.float64), 1.0, EPS)
    got = np64(r.rstd)
    fine = [0, 1, 2, 5, 6, 7]
    # a reciprocal root below 2^-126 keeps fewer digits
    assert np.all(np.abs(got[fine] - rstd[fine]) <= 1.01 * U * rstd[fine] + 2.0 ** -149)
    assert got[3] == 0 and np.isnan(got[4])
    out = np64(r.y)
    within(out[fine], y[fine], 3.1 * U * np.abs(y[fine]) + np.abs(x[fine]) * 2.0 ** -149)
    assert not out[0].any()
    assert np.isnan(out[3, 5]) and not np.delete(out[3], 5).any() and np.isnan(out[4]).all()
    stored = np64(pc.pc_q8_load(r.q, torch.float32))
    assert np.isnan(stored[4]).all() and np.isnan(stored[3, 5]) and not np.delete(stored[3], 5).any()


def test_norm_counts_over_many_rows():
    rng = np.random.default_rng(21)
    for rows, cols in ((3000, 72), (700, 2056), (300, 16392), (40, 33000)):
        x = activation(rng, rows, cols, "bf16")
        counts = torch.zeros(256, dtype=torch.int64, device=DEV)
        a = pc.pc_rmsnorm_store(x, format="int8", counts=counts)
        b = pc.pc_rmsnorm_store(x, format="int8")
        assert torch.equal(a.q.symbols, b.q.symbols) and torch.equal(a.q.scales, b.q.scales) and torch.equal(a.rstd, b.rstd)
        assert torch.equal(counts, torch.bincount(a.q.symbols.view(-1).long(), minlength=256))


def test_norm_of_strided_rows_writes_only_its_own():
    rng = np.random.default_rng(22)
    for cols in (40, 1000, 1003, 4104):
        wide = activation(rng, 9, cols + 13, "bf16")
        x, res = wide[:, 5:5 + cols], activation(rng, 9, cols + 3, "f32")[:, 3:]
        total = torch.full((9, cols + 8), 5.0, device=DEV)
        mask = pc.DropoutMask(0.2, 4)
        a = pc.pc_rmsnorm_store(x, residual=res, mask=mask, sum_out=total[:, 2:2 + cols], y="plain")
        b = pc.pc_rmsnorm_store(x.contiguous(), residual=res.contiguous(), mask=mask, y="plain")
        assert torch.equal(a.sum, b.sum) and torch.equal(a.y, b.y) and torch.equal(a.q.symbols, b.q.symbols)
        assert bool((total[:, :2] == 5).all()) and bool((total[:, 2 + cols:] == 5).all())
        dy = activation(rng, 9, cols + 1, "bf16")[:, 1:]
        ds = activation(rng, 9, cols + 2, "f32")[:, :cols]
        w = torch.ones(cols, device=DEV)
        g = pc.pc_rmsnorm_backward(dy, a.sum, w, a.rstd, d_sum=ds, mask=mask)
        h = pc.pc_rmsnorm_backward(dy.contiguous(), b.sum, w, b.rstd, d_sum=ds.contiguous(), mask=mask)
        assert torch.equal(g.residual, h.residual) and torch.equal(g.x, h.x) and torch.equal(g.weight, h.weight)
        # x as the sum's place, and several leading dimensions
        c = pc.pc_rmsnorm_store(b.y.view(3, 3, cols).clone(), mask=mask)
        z = b.y.clone()
        d = pc.pc_rmsnorm_store(z, mask=mask, sum_out=z)
        assert c.sum.shape == (3, 3, cols) and c.rstd.shape == (3, 3)
        assert d.sum is z and torch.equal(c.sum.view(9, cols), z) and torch.equal(c.q.symbols, d.q.symbols)


def test_norm_stored_views():
    rng = np.random.default_rng(23)
    sym, codes = q8.store(rng.normal(size=(6, 256)), "e4m3")
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV))
    part = q.columns(64, 200 // 32 * 32 + 32)
    dy = activation(rng, 6, part.shape[1], "bf16")
    rstd, w = torch.rand(6, device=DEV), torch.rand(part.shape[1], device=DEV)
    dense = pc.Q8(part.symbols.contiguous(), part.scales.contiguous())
    a, b = pc.pc_rmsnorm_backward(dy, part, w, rstd), pc.pc_rmsnorm_backward(dy, dense, w, rstd)
    assert torch.equal(a.residual, b.residual) and torch.equal(a.weight, b.weight)


def test_norm_weight_gradient_without_rows():
    w = torch.rand(50, device=DEV)
    none = torch.empty(0, 50, device=DEV)
    r = pc.pc_rmsnorm_backward(none, none, w, torch.empty(0, device=DEV))
    assert r.residual.shape == (0, 50) and not bool(r.weight.any())
    old = torch.rand(50, device=DEV)
    r = pc.pc_rmsnorm_backward(none, none, w, torch.empty(0, device=DEV), weight_out=old.clone(), accumulate=True)
    assert torch.equal(r.weight, old)
    s = pc.pc_rmsnorm_store(none, w, residual=none)
    assert s.sum.shape == (0, 50) and s.q.symbols.shape == (0, 50)


# sizes on both sides of every change of launch: units a lane, parts of waves, ragged and whole widths,
# streamed inputs, rows read twice, several rows of a team
LAUNCHES = [(5, 128), (5, 136), (70, 256), (70, 264), (5, 512), (5, 520), (1300, 64), (1300, 250), (9, 8192), (9, 8200),
            (3, 16384), (3, 16392), (3, 16390), (3, 32768), (3, 32776), (9000, 72), (1100, 512), (700, 520), (300, 1003),
            (512, 8192), (513, 4096), (512, 4104), (512, 40), (513, 40), (1, 65), (37, 8192)]


@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_norm_where_launches_change(dtype, res):
    rng = np.random.default_rng(24)
    for rows, cols in LAUNCHES:
        say("norm launches", rows, cols, dtype, res)
        x, residual = activation(rng, rows, cols, dtype), activation(rng, rows, cols, res)
        w = torch.rand(cols, device=DEV) + 0.5
        mask = pc.DropoutMask(0.1, 3)
        r = pc.pc_rmsnorm_store(x, w, residual, mask, y="plain")
        total = step.dropout(np64(x), 0.1, 3, 0)
        within(np64(r.sum), total + np64(residual), 3 * U * (np.abs(total) + np.abs(np64(residual))), res)
        h = np64(r.sum)
        y, rstd = step.norm(h, np64(w), EPS)
        assert np.all(np.abs(np64(r.rstd) - rstd) <= 1.01 * U * rstd)
        within(np64(r.y), y, 3.1 * U * np.abs(y), dtype)
        pick = np.unique(np.r_[0, rows // 2, rows - 1])
        check_stored(pc.Q8(r.q.symbols[pick].contiguous(), r.q.scales[pick].contiguous()), y[pick], "e4m3")
        dy = activation(rng, rows, cols, dtype)
        g = pc.pc_rmsnorm_backward(dy, r.sum, w, r.rstd, d_sum=residual, mask=mask)
        check_backward(g, dy, h, w, r.rstd, residual, dtype, res, 0.1)


def check_backward(g, dy, h, w, rstd, ds, dtype, res, p):
    rows, cols = h.shape
    d, dw = step.norm_backward(np64(dy), h, np64(w), np64(rstd), np64(ds))
    r64 = np64(rstd)[:, None]
    n, gw = h * r64, np64(dy) * np64(w)
    depth = 64 + cols / 1024
    tol = U * (r64 * (6 * np.abs(gw) + (depth + 8) * np.abs(n) * np.abs(gw * n).mean(1, keepdims=True))
               + 2 * np.abs(np64(ds)) + 2 * np.abs(d))
    within(np64(g.residual), d, tol, res)
    keep = 65536 / (65536 - step.below(p))
    within(np64(g.x), step.dropout(d, p, 3, 0), keep * (tol + 3 * U * np.abs(d)), dtype)
    within(np64(g.weight), dw, (rows + 40) * U * np.abs(np64(dy) * n).sum(0))


def test_norm_of_large_inputs():
    """Inputs of 256 MiB and more, which the kernels stream, against the same rows in small calls; rows past 2^31 elements."""
    rng = torch.Generator(device=DEV).manual_seed(5)
    for rows, cols, kind in ((8192, 8192, "bf16"), (33000, 2048, "bf16"), (4100, 8192, "f32"), (4200, 16384, "f16"),
                             (131073, 16400, "bf16")):
        say("large norm", rows, cols, kind)
        x = torch.randn(rows, cols, generator=rng, device=DEV, dtype=DT[kind])
        res = x if cols == 16400 else torch.randn(rows, cols, generator=rng, device=DEV, dtype=DT[kind])
        w = torch.rand(cols, device=DEV) + 0.5
        r = pc.pc_rmsnorm_store(x, w, res)
        g = pc.pc_rmsnorm_backward(x, r.sum, w, r.rstd, d_sum=res)
        for first in (0, rows // 2, rows - 40):
            part = slice(first, first + 40)
            s = pc.pc_rmsnorm_store(x[part], w, res[part])
            assert torch.equal(s.sum, r.sum[part]) and torch.equal(s.q.symbols, r.q.symbols[part])
            assert torch.equal(s.q.scales, r.q.scales[part])
            # sums of squares in 64 bits may be added in another order, and rounded once
            assert bool(((s.rstd - r.rstd[part]).abs() <= 2.0 ** -23 * s.rstd).all())
            h = np64(s.sum)
            d, _ = step.norm_backward(np64(x[part]), h, np64(w), np64(r.rstd[part]), np64(res[part]))
            n, gw = h * np64(r.rstd[part])[:, None], np64(x[part]) * np64(w)
            tol = U * (np64(r.rstd[part])[:, None] * (6 * np.abs(gw) + 90 * np.abs(n) * np.abs(gw * n).mean(1, keepdims=True))
                       + 2 * np.abs(np64(res[part])) + 2 * np.abs(d))
            within(np64(g.residual[part]), d, tol, kind)
        del x, res, r, g


# -- log probabilities ---------------------------------------------------------

def check_row_results(x, r, tokens, scale, top, d_extra=0.0):
    x64, s64 = np64(x), float(np.float32(scale))
    rows, vocab = x64.shape
    logp, entropy, index, top_logp = step.logprobs(x64, tokens, s64, top)
    left = ~np.isneginf(x64).all(1)
    y, log_s, d = spread(np.where(left[:, None], x64, 0.0), s64, entropy, vocab)
    got = np64(r.logp).reshape(tokens.shape)
    for a, b, at in ((got, logp, tokens), (np64(r.top_logp) if top else None, top_logp, index)):
        if a is None:
            continue
        with np.errstate(over="ignore"):
            dead = np.isneginf(b.astype(np.float32))  # also what 32 bits cannot hold: 2 (-3.4e38 - 8) rounds to -infinity
        assert np.array_equal(np.isneginf(a), dead)
        inside = (at >= 0) & (at < vocab)
        yy = np.take_along_axis(y, np.where(inside, at, 0), 1)
        tol = d[:, None] + 4 * U * (np.abs(np.where(dead, 0, yy)) + np.abs(np.where(dead, 0, b)))
        within(np.where(dead, 0, a), np.where(dead, 0, b), np.where(dead, 0, tol))
    within(np64(r.entropy), entropy, (3 * d + 20 * U) * (1 + entropy + np.abs(log_s)))
    if top:
        assert np.array_equal(r.top_index.cpu().numpy(), index)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_logits(dtype):
    """Masks by -infinity and by the type's lowest value, that leave some, one or no token."""
    rng = np.random.default_rng(31)
    for vocab in (5, 300, 4099, 20000):
        for value in (-INF, LOWEST[dtype]):
            say("masked", dtype, vocab, value)
            x, _ = logits(rng, 6, vocab, dtype)
            x[1, : vocab // 2] = value
            x[2, 1:] = value
            x[3] = value
            x[4, 2:] = value
            x[5, vocab - 1:] = value
            tokens = np.stack([np.zeros(6, dtype=np.int64), np.full(6, vocab - 1), np.full(6, vocab // 3)], 1)
            t = torch.from_numpy(tokens).to(DEV)
            for scale in (1.0, 0.5, 2.0):
                r = pc.pc_logprobs(x, t, top=min(vocab, 20), scale=scale)
                check_row_results(x, r, tokens, scale, min(vocab, 20))
                d = torch.ones(6, 3, device=DEV)
                de = torch.ones(6, device=DEV)
                g = np64(pc.pc_logprobs_backward(x, r.stats, t, d, d_entropy=de, scale=scale))
                want = step.logprobs_backward(np64(x), tokens, scale, np.ones((6, 3)), np.ones(6))
                assert np.isfinite(g).all()
                # by components: the probabilities' errors and the output's rounding, generously 64 u each way
                size = scale * 4 * (1 + np.abs(np64(r.entropy)))[:, None] * 64 * U * max(1.0, vocab / 64)
                within(g, want, size, dtype)
                if value == -INF:
                    assert not g[3].any()


def test_rows_with_nothing_left():
    x = torch.full((3, 1000), -INF, device=DEV)
    t = torch.tensor([0, 999, -1], device=DEV)
    r = pc.pc_logprobs(x, t, top=4)
    assert r.logp.tolist() == [-INF, -INF, 0.0] and r.entropy.tolist() == [0.0] * 3
    assert r.top_index.tolist() == [[0, 1, 2, 3]] * 3 and bool(torch.isneginf(r.top_logp).all()) and bool(torch.isneginf(r.lse).all())
    g = pc.pc_logprobs_backward(x, r.stats, t, torch.ones(3, device=DEV), d_entropy=torch.ones(3, device=DEV))
    assert not bool(g.any())


@pytest.mark.parametrize("vocab", [40, 3001, 50000])
def test_nan_and_infinity_stay_visible(vocab):
    x = torch.randn(5, vocab, device=DEV)
    x[0, 7] = NAN
    x[1, 8] = INF
    x[2] = NAN
    x[3, 9] = -INF
    t = torch.zeros(5, dtype=torch.int64, device=DEV)
    r = pc.pc_logprobs(x, t, top=5)
    for v in (r.logp, r.entropy, r.lse, r.top_logp[:, 0]):
        assert torch.isnan(v).tolist() == [True, True, True, False, False]
    assert r.top_index[2].tolist() == [0, 1, 2, 3, 4] and int(r.top_index[1, 0]) == 8
    best = torch.where(torch.isnan(x[0]), -INF, x[0]).topk(5).indices
    assert r.top_index[0].tolist() == best.tolist()
    d = torch.ones(5, device=DEV)
    g = pc.pc_logprobs_backward(x, r.stats, t, d)
    assert torch.isnan(g).any(1).tolist() == [True, True, True, False, False]
    # rows without a gradient of their own get zeros, whatever their logits
    d[:3] = 0
    g = pc.pc_logprobs_backward(x, r.stats, t, d, d_entropy=torch.zeros(5, device=DEV))
    assert not bool(g[:3].any()) and bool(torch.isfinite(g).all()) and bool(g[4].any())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(2, 64), (1, 70), (3, 2048), (2, 9000), (1, 131072), (300, 5000), (4500, 600),
                                        (257, 33000)])
def test_equal_logits_go_by_index(dtype, rows, vocab):
    """Ties: constant rows, rows of few values, both zeros, ascending and descending ones."""
    rng = np.random.default_rng(32)
    top = min(64, vocab)
    for kind in range(5):
        say("ties", dtype, rows, vocab, kind)
        if kind == 0:
            x = np.full((rows, vocab), 1.5)
        elif kind == 1:
            x = rng.integers(0, 3, size=(rows, vocab)).astype(float)
        elif kind == 2:
            x = np.where(rng.random((rows, vocab)) < 0.5, 0.0, -0.0)
        else:
            x = np.tile(np.arange(vocab) % 1000 / 8.0, (rows, 1))
            x = x[:, ::-1] if kind == 4 else x
        t = tensor(x.astype(np.float32), dtype)
        r = pc.pc_logprobs(t, top=top)
        want = np.argsort(-np64(t), axis=1, kind="stable")[:, :top]
        assert np.array_equal(r.top_index.cpu().numpy(), want)


def test_top_of_one_and_of_all():
    rng = np.random.default_rng(33)
    for vocab in (1, 2, 63, 64):
        x, _ = logits(rng, 4, vocab, "bf16")
        for top in {1, vocab}:
            r = pc.pc_logprobs(x, top=top)
            assert np.array_equal(r.top_index.cpu().numpy(), np.argsort(-np64(x), axis=1, kind="stable")[:, :top])
            assert float(r.top_logp.max()) <= 0.0
    one = pc.pc_logprobs(torch.randn(3, 1, device=DEV) * 40, torch.zeros(3, dtype=torch.int64, device=DEV))
    # one exponential of what the rounded reference lost and its logarithm: within the bound of ln S, (1/64 + 70) u
    assert float(one.logp.max()) <= 0.0 and float(one.logp.min()) >= -71 * U and float(one.entropy.abs().max()) <= 233 * U


@pytest.mark.parametrize("shift", [-(1 << 13), 1 << 13, 1 << 20, -(1 << 30), 1 << 31])
def test_a_shift_of_all_logits(shift):
    """Probabilities depend on differences alone.  Logits are whole steps, so the shifted ones are exact."""
    rng = np.random.default_rng(35)
    unit = max(2.0 ** -8, abs(shift) * 2.0 ** -22)
    x = np.round(rng.normal(size=(4, 3000)) * 3 / unit) * unit
    x[:, 17] = np.ceil(10 / unit) * unit
    tokens = np.array([[17, 0], [1, 2], [2999, 17], [5, 5]])
    t = torch.from_numpy(tokens).to(DEV)
    scale = 0.75
    s = torch.from_numpy((x + shift).astype(np.float32)).to(DEV)
    assert np.array_equal(np64(s) - shift, x)
    r = pc.pc_logprobs(s, t, top=8, scale=scale)
    check_row_results(torch.from_numpy(x.astype(np.float32)).to(DEV), r, tokens, scale, 8)
    d, de = rng.normal(size=(4, 2)).astype(np.float32), rng.normal(size=4).astype(np.float32)
    g = np64(pc.pc_logprobs_backward(s, r.stats, t, torch.from_numpy(d).to(DEV), torch.from_numpy(de).to(DEV), scale=scale))
    want = step.logprobs_backward(x, tokens, scale, d.astype(np.float64), de.astype(np.float64))
    logp = step.log_softmax(x, scale)
    p = np.exp(logp)
    entropy = -(p * np.where(p > 0, logp, 0)).sum(1, keepdims=True)
    _, _, off = spread(x, scale, entropy[:, 0], 3000)
    # a probability is off as its logarithm is (d of ln S, twice 8 u |logp|), the entropy by 3 d (1 + ...)
    size = np.abs(d).sum(1, keepdims=True) + np.abs(de)[:, None] * (np.abs(logp) + 2 * entropy + 2)
    tol = p * size * (4 * off[:, None] + 16 * U * (1 + np.abs(logp))) + (np.abs(want) > p * size * 2) * 8 * U * size
    within(g, want, tol)


def test_tokens_outside_and_padding():
    x = torch.randn(2, 50, device=DEV)
    tokens = torch.tensor([[3, -100, 49, 3], [50, -1, 1 << 40, -(1 << 40)]], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = pc.pc_logprobs(x, tokens, padding=-100, status=status)
    assert int(status) == pc.PC_ERR_INVALID_ARG
    assert r.logp[1].tolist() == [0.0] * 4 and float(r.logp[0, 1]) == 0.0 and bool((r.logp[0, [0, 2, 3]] < 0).all())
    d = torch.full((2, 4), NAN, device=DEV)
    d[0] = torch.tensor([1.0, NAN, 2.0, 3.0])
    g = np64(pc.pc_logprobs_backward(x, r.stats, tokens, d, padding=-100))
    want = step.logprobs_backward(np64(x), tokens.cpu().numpy(), 1.0, np.array([[1.0, 0, 2, 3], [0] * 4]), np.zeros(2), -100)
    within(g, want, 200 * U)
    assert not g[1].any()
    status.zero_()
    pc.pc_logprobs(x, torch.tensor([[3], [-100]], device=DEV), padding=-100, status=status)
    assert int(status) == 0


def test_logits_of_other_shapes_and_strides():
    rng = np.random.default_rng(34)
    for vocab in (100, 6007, 40000):
        wide, _ = logits(rng, 6, vocab + 11, "bf16")
        x = wide[:, 3:3 + vocab]
        tokens = torch.from_numpy(rng.integers(0, vocab, size=(6, 2))).to(DEV)
        a, b = pc.pc_logprobs(x, tokens, top=9), pc.pc_logprobs(x.contiguous(), tokens, top=9)
        assert torch.equal(a.logp, b.logp) and torch.equal(a.stats, b.stats) and torch.equal(a.top_index, b.top_index)
        c = pc.pc_logprobs(x.contiguous().view(2, 3, vocab), tokens.view(2, 3, 2), top=9)
        assert c.logp.shape == (2, 3, 2) and c.entropy.shape == (2, 3) and c.top_logp.shape == (2, 3, 9)
        assert torch.equal(c.logp.view(6, 2), a.logp) and torch.equal(c.entropy.reshape(6), a.entropy)
        one = pc.pc_logprobs(x[0], tokens[0, 0])
        assert one.logp.shape == () and one.entropy.shape == () and float(one.entropy) == float(a.entropy[0])
        d = torch.randn(6, 2, device=DEV)
        out = torch.full((6, vocab + 5), 7.0, dtype=torch.bfloat16, device=DEV)
        g = pc.pc_logprobs_backward(x.contiguous(), b.stats, tokens, d)
        pc.pc_logprobs_backward(x, a.stats, tokens, d, out=out[:, 2:2 + vocab])
        assert torch.equal(out[:, 2:2 + vocab], g)
        assert bool((out[:, :2] == 7).all()) and bool((out[:, 2 + vocab:] == 7).all())
        h = pc.pc_logprobs_backward(x.contiguous(), b.stats, d_entropy=torch.ones(6, device=DEV))
        assert h.shape == (6, vocab)
    none = torch.empty(0, 30, device=DEV)
    r = pc.pc_logprobs(none, torch.empty(0, 2, dtype=torch.int64, device=DEV), top=3)
    assert r.logp.shape == (0, 2) and r.top_index.shape == (0, 3) and r.entropy.shape == (0,)
    assert pc.pc_logprobs_backward(none, r.stats, torch.empty(0, 2, dtype=torch.int64, device=DEV),
                                   torch.empty(0, 2, device=DEV)).shape == (0, 30)


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 4096, 2048), ("bf16", 4095, 2048), ("bf16", 4096, 32776),
                                              ("bf16", 257, 33000), ("bf16", 256, 16384), ("bf16", 256, 16376),
                                              ("f32", 255, 8192), ("f32", 255, 8188), ("bf16", 4200, 16000),
                                              ("f32", 600, 60001), ("f16", 20, 260000), ("f32", 512, 16384),
                                              ("f32", 512, 16380), ("f32", 513, 49148), ("bf16", 513, 98304),
                                              ("bf16", 100, 170000), ("bf16", 2, 5600000)])
def test_logprobs_where_launches_change(dtype, rows, vocab):
    rng = torch.Generator(device=DEV).manual_seed(6)
    x = (torch.randn(rows, vocab, generator=rng, device=DEV) * 3).to(DT[dtype])
    tokens = torch.randint(0, vocab, (rows, 2), generator=rng, device=DEV)
    r = pc.pc_logprobs(x, tokens, top=20)
    pick = torch.tensor(sorted({0, 1, rows // 2, rows - 1}), device=DEV)
    x64, t = x[pick], tokens[pick].cpu().numpy()
    part = pc.LogProbs(r.logp[pick], r.top_index[pick], r.top_logp[pick], r.stats[pick].contiguous(), (len(pick),))
    check_row_results(x64, part, t, 1.0, 20)
    d = torch.randn(rows, 2, generator=rng, device=DEV)
    g = pc.pc_logprobs_backward(x, r.stats, tokens, d)
    h = pc.pc_logprobs_backward(x64.contiguous(), part.stats, tokens[pick], d[pick])
    assert torch.equal(g[pick], h)
    assert torch.equal(pc.pc_logprobs(x, tokens).stats, r.stats)


def test_logits_past_2_to_the_31():
    rows, vocab = 33000, 65600  # 2^31 elements are passed in row 32736
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device=DEV)
    x[:, 5] = 3.0
    x[32737:, 77] = 9.0
    t = torch.full((rows,), 77, device=DEV)
    r = pc.pc_logprobs(x, t, top=2)
    assert r.top_index[0].tolist() == [5, 0] and r.top_index[-1].tolist() == [77, 5]
    d = torch.ones(rows, device=DEV)
    pc.pc_logprobs_backward(x, r.stats, t, d, out=x)
    for i in (0, 32736, 32737, rows - 1):
        z = np.zeros((1, vocab))
        z[0, 5] = 3.0
        z[0, 77] = 9.0 if i >= 32737 else 0.0
        want = step.logprobs_backward(z, np.array([[77]]), 1.0, np.ones((1, 1)), np.zeros(1))
        within(np64(x[i:i + 1]), want, 2000 * U * np.abs(want) + 4 * U, "bf16")


# -- streams and graphs ------------------------------------------------------------

def test_on_another_stream():
    rng = np.random.default_rng(41)
    x = activation(rng, 300, 1000, "bf16")
    tokens = torch.from_numpy(rng.integers(0, 1000, size=300)).to(DEV)
    w = torch.rand(1000, device=DEV)
    mask = pc.DropoutMask(0.3, 8)

    def everything():
        n = pc.pc_rmsnorm_store(x, w, x, mask, y="plain")
        g = pc.pc_rmsnorm_backward(n.y, n.sum, w, n.rstd, d_sum=x, mask=mask)
        p = pc.pc_logprobs(n.y, tokens, top=5)
        b = pc.pc_logprobs_backward(n.y, p.stats, tokens, p.logp)
        return n.sum, n.y, n.q.symbols, n.rstd, g.residual, g.x, g.weight, p.logp, p.top_index, p.stats, b, pc.pc_dropout(x, mask)

    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    """A captured step draws a new mask where the state on the device changes, and equals the eager one each time."""
    rng = np.random.default_rng(42)
    x, res = activation(rng, 130, 264, "bf16"), activation(rng, 130, 264, "f32")
    w = torch.rand(264, device=DEV)
    big = activation(rng, 2, 20000, "f32")
    tokens = torch.from_numpy(rng.integers(0, 264, size=(130, 3))).to(DEV)
    few = torch.from_numpy(rng.integers(0, 20000, size=2)).to(DEV)
    state = torch.tensor([99, 0], device=DEV)
    mask = pc.DropoutMask(0.4, state, offset=5)

    def everything():
        n = pc.pc_rmsnorm_store(x, w, res, mask, y="stored")
        g = pc.pc_rmsnorm_backward(n.y, n.sum, w, n.rstd, d_sum=res, mask=mask)
        p = pc.pc_logprobs(n.y, tokens, top=7)
        b = pc.pc_logprobs_backward(n.y, p.stats, tokens, p.logp, d_entropy=p.logp[:, 0].contiguous())
        s = pc.pc_logprobs(big, few, top=7)
        return [n.sum, n.y, n.q.symbols, g.residual, g.x, g.weight, p.logp, p.top_index, b, s.logp, s.top_index, s.stats,
                pc.pc_dropout(x, mask)]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything()
    seen = []
    for k in range(4):
        state.copy_(torch.tensor([99 + k // 2, k]))
        big.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, everything()):
            assert torch.equal(a, b)
        seen.append(got[-1])
    assert not any(torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    f, w = torch.zeros(4, device=DEV), torch.zeros(64, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    m = pc.DropoutMask(0.1)
    bad = [
        (TypeError, lambda: pc.pc_dropout(x, None)), (TypeError, lambda: pc.pc_dropout(x, 0.1)),
        (TypeError, lambda: pc.pc_dropout(x, m, out=x.float())), (ValueError, lambda: pc.pc_dropout(x, m, out=x[:3])),
        (ValueError, lambda: pc.pc_dropout(x.t(), m)), (ValueError, lambda: pc.pc_dropout(f[0], m)),
        (TypeError, lambda: pc.DropoutMask(0.1, t)), (TypeError, lambda: pc.DropoutMask(0.1, t.int()[:2])),
        (ValueError, lambda: pc.pc_rmsnorm_store(x, w[:63])), (TypeError, lambda: pc.pc_rmsnorm_store(x, w.double())),
        (ValueError, lambda: pc.pc_rmsnorm_store(x, torch.zeros(128, device=DEV)[::2])),
        (TypeError, lambda: pc.pc_rmsnorm_store(x, residual=x.half())), (ValueError, lambda: pc.pc_rmsnorm_store(x, residual=x[:2])),
        (ValueError, lambda: pc.pc_rmsnorm_store(x, sum_out=x)), (ValueError, lambda: pc.pc_rmsnorm_store(x, format="e5m2")),
        (ValueError, lambda: pc.pc_rmsnorm_store(x, format=None, y="stored")), (ValueError, lambda: pc.pc_rmsnorm_store(x, y="f32")),
        (ValueError, lambda: pc.pc_rmsnorm_store(x, format=None, counts=torch.zeros(256, dtype=torch.int64, device=DEV))),
        (TypeError, lambda: pc.pc_rmsnorm_store(x, counts=t)), (TypeError, lambda: pc.pc_rmsnorm_store(x, mask=0.5)),
        (TypeError, lambda: pc.pc_rmsnorm_store(x, residual=x, sum_out=x.float())),
        (pc.PcError, lambda: pc.pc_rmsnorm_store(x, eps=0.0)), (pc.PcError, lambda: pc.pc_rmsnorm_store(x, eps=NAN)),
        (TypeError, lambda: pc.pc_rmsnorm_store(x, y="plain", dtype=torch.float64)),
        (TypeError, lambda: pc.pc_rmsnorm_backward(x, x.half(), w, f)), (TypeError, lambda: pc.pc_rmsnorm_backward(x, x, w, t)),
        (TypeError, lambda: pc.pc_rmsnorm_backward(x, x, w, f[:3])), (TypeError, lambda: pc.pc_rmsnorm_backward(x, x, w, f, d_sum=x.float())),
        (ValueError, lambda: pc.pc_rmsnorm_backward(x, x, None, f, weight_out=w)),
        (ValueError, lambda: pc.pc_rmsnorm_backward(x, x, w, f, accumulate=True)),
        (TypeError, lambda: pc.pc_rmsnorm_backward(x, x, w, f, weight_out=w.half())),
        (ValueError, lambda: pc.pc_rmsnorm_backward(x, x, w, f, weight_out=w[:5])),
        (ValueError, lambda: pc.pc_rmsnorm_backward(x, x[:2], w, f)),
        (ValueError, lambda: pc.pc_rmsnorm_backward(x, pc.pc_q8_store(x[:2]), w, f)),
        (TypeError, lambda: pc.pc_rmsnorm_backward(x, pc.pc_q8_store(x), w, f, dtype=torch.float16)),
        (TypeError, lambda: pc.pc_logprobs(x, f)), (ValueError, lambda: pc.pc_logprobs(x, t[:3])),
        (ValueError, lambda: pc.pc_logprobs(x, t.cpu())), (ValueError, lambda: pc.pc_logprobs(x, top=-1)),
        (pc.PcError, lambda: pc.pc_logprobs(x, top=65)), (pc.PcError, lambda: pc.pc_logprobs(x[:, :5], top=6)),
        (pc.PcError, lambda: pc.pc_logprobs(x, scale=0.0)), (pc.PcError, lambda: pc.pc_logprobs(x, t.view(4, 1).expand(4, 65))),
        (TypeError, lambda: pc.pc_logprobs(x, t, status=t)),
        (TypeError, lambda: pc.pc_logprobs_backward(x, f, t, f)), (ValueError, lambda: pc.pc_logprobs_backward(x, torch.zeros(4, 4, device=DEV), t)),
        (TypeError, lambda: pc.pc_logprobs_backward(x, torch.zeros(4, 4, device=DEV), t, f.half())),
        (ValueError, lambda: pc.pc_logprobs_backward(x, torch.zeros(4, 4, device=DEV), t, f[:3])),
        (ValueError, lambda: pc.pc_logprobs_backward(x, torch.zeros(4, 4, device=DEV), d_entropy=f[:3])),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            raise AssertionError("call %d passed" % k)


# -- forms that only the C entries have ------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(70, 264), (512, 8192), (400, 5001), (600, 520), (9, 8200), (5, 8191), (4, 33000), (3, 40001)])
def test_norm_backward_in_place(rows, cols):
    """The residual's gradient over the one that comes in, x's over y's."""
    lib = pc._lib.lib
    rng = np.random.default_rng(51)
    dy, h, ds = (activation(rng, rows, cols, "bf16") for _ in range(3))
    w, rstd = torch.rand(cols, device=DEV), torch.rand(rows, device=DEV)
    mask = pc.DropoutMask(0.3, 4)
    want = pc.pc_rmsnorm_backward(dy, h, w, rstd, d_sum=ds, mask=mask)
    need = pc.pc_rmsnorm_backward_workspace_bytes(rows, cols)
    ws, dw = torch.empty(need, dtype=torch.uint8, device=DEV), torch.empty(cols, device=DEV)
    st = lib.pc_rmsnorm_backward(dy.data_ptr(), pc.PC_BF16, rows, cols, cols, h.data_ptr(), pc.PC_BF16, cols, None,
                                 w.data_ptr(), pc.PC_F32, rstd.data_ptr(), ds.data_ptr(), cols, mask.arg, ds.data_ptr(), cols,
                                 dy.data_ptr(), cols, dw.data_ptr(), pc.PC_F32, 0, ws.data_ptr(), need,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == pc.PC_OK
    assert torch.equal(ds, want.residual) and torch.equal(dy, want.x) and torch.equal(dw, want.weight)


@pytest.mark.parametrize("rows,cols", [(70, 264), (5, 8191), (3, 40001), (300, 96)])
def test_norm_without_its_sum(rows, cols):
    """A last norm, whose sum nothing reads: the same y; and a call that wants nothing but rstd."""
    lib = pc._lib.lib
    rng = np.random.default_rng(52)
    x, res = activation(rng, rows, cols, "f16"), activation(rng, rows, cols, "f32")
    mask = pc.DropoutMask(0.3, 4)
    want = pc.pc_rmsnorm_store(x, None, res, mask, y="plain")
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    st = lib.pc_rmsnorm_store(x.data_ptr(), pc.PC_F16, rows, cols, cols, res.data_ptr(), pc.PC_F32, cols, mask.arg, None, 0,
                              1e-6, None, 0, 0, None, None, None, y.data_ptr(), pc.PC_F16, cols, 0, None, stream)
    assert st == pc.PC_OK and torch.equal(y, want.y)
    st = lib.pc_rmsnorm_store(x.data_ptr(), pc.PC_F16, rows, cols, cols, res.data_ptr(), pc.PC_F32, cols, mask.arg, None, 0,
                              1e-6, None, 0, 0, None, None, None, None, 0, 0, 0, rstd.data_ptr(), stream)
    assert st == pc.PC_OK and torch.equal(rstd, want.rstd)
    bare = pc.pc_rmsnorm_store(x, residual=res, mask=mask, format=None)
    assert bare.q is None and bare.y is None and torch.equal(bare.sum, want.sum)


def test_masked_stretches_and_alternatives():
    """Splits that are masked throughout, with more alternatives than the rest of the row has tokens."""
    for vocab, left in ((40000, 3), (40000, 30), (150001, 10), (9000, 64)):
        x = torch.full((3, vocab), -INF, device=DEV)
        at = torch.linspace(0, vocab - 1, left, device=DEV).long()
        x[0, at] = torch.arange(left, device=DEV, dtype=torch.float32)
        x[1, vocab // 2:vocab // 2 + left] = 1.0
        x[2, -left:] = torch.randn(left, device=DEV)
        r = pc.pc_logprobs(x, top=64)
        assert np.array_equal(r.top_index.cpu().numpy(), np.argsort(-np64(x), axis=1, kind="stable")[:, :64]), (vocab, left)
