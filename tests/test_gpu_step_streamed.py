"""The variants that inputs past the memory-side cache take, over all of their rows:
64-bit forms on the device, by blocks of rows.

Tolerances, with u = 2^-24 and the terms of test_gpu_step.py.  The weight's
gradient is bounded by the additions that a term really passes: the rows that one
lane takes (workgroups are 256 at least, so rows / 256 + 1), up to 16 teams of a
workgroup, a 64th of up to 2048 partial sums (32), and the 64 groups of the
join; each is off by u of what is summed, 4 u more for the term itself.  (Rows
that are read twice have 48 partial sums or more here, so rows / 48, but no teams
and one turn of the join: less.)  A lost row of thousands is far above that."""
import numpy as np
import pytest
import torch

from oracle import q8, step
from test_gpu_step import DEV, DT, EPS, HALF_STEP, TINY, U, check_stored, np64, say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc

BLOCK = 1024


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def numbers(first, rows, cols, seed, offset, device=None):
    """The 16 bits of rows [first, first + rows), in 64-bit integers that wrap."""
    word, device = 0xFFFFFFFF, device or DEV
    block = torch.arange(-(-cols // 8), device=device).expand(rows, -1)
    row = torch.arange(first, first + rows, device=device).unsqueeze(1).expand(block.shape)
    c = block, row, torch.full_like(block, offset & word), torch.full_like(block, offset >> 32)
    k0, k1 = seed & word, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = ((b >> 32) & word) ^ c[1] ^ k0, b & word, ((a >> 32) & word) ^ c[3] ^ k1, a & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    words = torch.stack(c, 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, -1)[:, :cols]


def check(got, want, tol, dtype):
    tol = tol + HALF_STEP[dtype] * want.abs() + TINY[dtype]
    off = (got.double() - want).abs() - tol
    assert bool(torch.isfinite(got).all()) and float(off.max()) <= 0, (float(off.max()), int((off > 0).sum()))


def test_numbers_of_the_device_are_those_of_the_host():
    want = step.numbers(40, 75, (7 << 32) | 5, (9 << 32) | 11)
    assert np.array_equal(numbers(0, 40, 75, (7 << 32) | 5, (9 << 32) | 11).cpu().numpy(), want)
    assert np.array_equal(numbers(33, 7, 75, (7 << 32) | 5, (9 << 32) | 11).cpu().numpy(), want[33:])


def kept_by(first, rows, cols, seed, offset, p):
    """What each element is multiplied by."""
    t = step.below(p)
    return torch.where(numbers(first, rows, cols, seed, offset) < t, 0.0, 65536 / (65536 - t)).double()


def rows_of(g, rows, cols, dtype, size=1.0):
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return (x * torch.exp(torch.randn(rows, 1, generator=g, device=DEV)) * size).to(DT[dtype])


@pytest.mark.parametrize("dtype,res,rows,cols,kept,p", [
    # two units a lane, and one, streamed: the sum stored in both forms or plain, with a mask and without
    ("bf16", "bf16", 6700, 8192, "e4m3", 0.1), ("bf16", "bf16", 6701, 8192, "int8", 0.0),
    ("f16", "f16", 3400, 16384, "e4m3", 0.25), ("bf16", "bf16", 5700, 8192, "plain", 0.25),
    ("bf16", "bf16", 13500, 4104, "e4m3", 0.1), ("f16", "f16", 27001, 2056, "int8", 0.25),
    ("bf16", "f32", 9400, 4096, "e4m3", 0.1), ("f16", "f32", 4800, 8192, "int8", 0.0), ("bf16", "f32", 6600, 4104, "plain", 0.25),
    ("f32", "f32", 7500, 4096, "e4m3", 0.1), ("f32", "f32", 2800, 8192, "plain", 0.25),
    # the same below the border, and of ragged widths, which do not stream
    ("bf16", "bf16", 6500, 8192, "e4m3", 0.1), ("bf16", "bf16", 6700, 8190, "e4m3", 0.1), ("f16", "f32", 6001, 4101, "int8", 0.1),
    # parts of waves, which do not either
    ("bf16", "bf16", 450001, 128, "e4m3", 0.1), ("bf16", "bf16", 220000, 256, "int8", 0.1),
    # rows read twice
    ("bf16", "bf16", 1400, 40008, "e4m3", 0.1), ("bf16", "f32", 2000, 16384, "int8", 0.25)])
def test_norm_gradients(dtype, res, rows, cols, kept, p):
    g = torch.Generator(device=DEV).manual_seed(rows)
    say("streamed gradient", dtype, res, rows, cols, kept, p)
    dy, ds = rows_of(g, rows, cols, dtype), rows_of(g, rows, cols, res)
    total = rows_of(g, rows, cols, res, 3.0)
    w = torch.rand(cols, generator=g, device=DEV) + 0.5
    mask = pc.DropoutMask(p, 11, 12) if p else None
    if kept == "plain":
        q, h_of = total, lambda part: total[part].double()
    else:
        q = pc.pc_q8_store(total, kept)
        table = torch.from_numpy(q8.elements(kept)).to(DEV)
        columns = torch.arange(cols, device=DEV) // 32
        h_of = lambda part: table[q.symbols[part].long()] * torch.exp2(q.scales[part].double() - 127)[:, columns]  # noqa: E731
    rstd = torch.cat([(h_of(slice(i, i + BLOCK)).square().mean(1) + EPS).rsqrt().float() for i in range(0, rows, BLOCK)])
    r = pc.pc_rmsnorm_backward(dy, q, w, rstd, d_sum=ds, mask=mask, dtype=DT[res])
    dw, size = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    depth = 64 + cols / 1024
    for i in range(0, rows, BLOCK):
        part = slice(i, min(rows, i + BLOCK))
        h, r64 = h_of(part), rstd[part].double()[:, None]
        n, gw, s = h * r64, dy[part].double() * w.double(), ds[part].double()
        d = r64 * (gw - n * (gw * n).mean(1, keepdim=True)) + s
        tol = U * (r64 * (6 * gw.abs() + (depth + 8) * n.abs() * (gw * n).abs().mean(1, keepdim=True)) + 2 * s.abs() + 2 * d.abs())
        check(r.residual[part], d, tol, res)
        if p:
            keep = kept_by(i, h.shape[0], cols, 11, 12, p)
            check(r.x[part], d * keep, keep * (tol + 3 * U * d.abs()), dtype)
        elif res == dtype:
            assert r.x is r.residual
        else:
            check(r.x[part], d, tol, dtype)
        terms = dy[part].double() * n
        dw += terms.sum(0)
        size += terms.abs().sum(0)
    check(r.weight, dw, (rows / 256 + 1 + 16 + 32 + 64 + 4) * U * size, "f32")


@pytest.mark.parametrize("dtype,res,rows,cols,p,fmt", [
    ("bf16", "bf16", 8300, 8192, 0.1, "e4m3"), ("bf16", "bf16", 8300, 8192, 0.0, "int8"), ("f16", "f16", 4200, 16384, 0.25, "int8"),
    ("bf16", None, 16500, 8192, 0.25, "e4m3"), ("bf16", "f32", 11000, 4096, 0.1, "e4m3"), ("f32", "f32", 8300, 4104, 0.1, "int8"),
    ("f32", "f32", 2100, 16384, 0.25, "e4m3"), ("bf16", "bf16", 2100, 32768, 0.1, "e4m3"), ("bf16", "bf16", 33000, 2048, 0.1, "e4m3"),
    # below the border, ragged, and rows read twice
    ("bf16", "bf16", 8100, 8192, 0.1, "e4m3"), ("bf16", "bf16", 8300, 8190, 0.1, "e4m3"), ("f16", "f32", 1100, 40008, 0.1, "int8"),
    ("bf16", "bf16", 530000, 128, 0.1, "e4m3")])
def test_norms(dtype, res, rows, cols, p, fmt):
    g = torch.Generator(device=DEV).manual_seed(rows)
    say("streamed norm", dtype, res, rows, cols, p, fmt)
    x = rows_of(g, rows, cols, dtype)
    residual = rows_of(g, rows, cols, res, 3.0) if res else None
    w = torch.rand(cols, generator=g, device=DEV) + 0.5
    mask = pc.DropoutMask(p, 21, 22) if p else None
    r = pc.pc_rmsnorm_store(x, w, residual, mask, format=fmt, y="plain")
    s = pc.pc_rmsnorm_store(x, w, residual, mask, format=fmt, y="stored", dtype=torch.bfloat16)
    assert torch.equal(s.sum, r.sum) and torch.equal(s.rstd, r.rstd)
    assert torch.equal(s.q.symbols, r.q.symbols) and torch.equal(s.q.scales, r.q.scales)
    assert torch.equal(s.y, pc.pc_q8_load(s.q, torch.bfloat16))
    for i in range(0, rows, BLOCK):
        part = slice(i, min(rows, i + BLOCK))
        h, n = x[part].double(), x[part].shape[0]
        if p:
            h = h * kept_by(i, n, cols, 21, 22, p)
        size = h.abs()
        if res:
            h, size = h + residual[part].double(), size + residual[part].double().abs()
        check(r.sum[part], h, 3 * U * size, res or dtype)
        h = r.sum[part].double()
        rstd = (h.square().mean(1) + EPS).rsqrt()
        assert bool(((r.rstd[part].double() - rstd).abs() <= 1.01 * U * rstd).all())
        y = h * rstd[:, None] * w.double()
        check(r.y[part], y, 3.1 * U * y.abs(), dtype)
        # the stored form: of each block some rows byte for byte, of all rows the values to half a step
        # (of e4m3 2^-4 of the value or 2^-10 of the scale; of int8 half the scale)
        scale = torch.exp2(r.q.scales[part].double() - 127).repeat_interleave(32, 1)[:, :cols]
        half = torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10) if fmt == "e4m3" else scale / 2
        stored = pc.pc_q8_load(pc.Q8(r.q.symbols[part], r.q.scales[part], fmt), torch.float32).double()
        assert bool(((stored - y).abs() <= half * (1 + 2.0 ** -20)).all())
        some = torch.tensor(sorted({0, n // 2, n - 1}), device=DEV)
        if i == 0 or i + BLOCK >= rows or i // BLOCK % 4 == 1:
            check_stored(pc.Q8(r.q.symbols[part][some].contiguous(), r.q.scales[part][some].contiguous(), fmt),
                         np64(y[some]), fmt)


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 4200, 16000), ("f32", 600, 60001), ("f16", 2100, 32003),
                                              # not streamed
                                              ("bf16", 4100, 16000), ("f32", 300, 60001)])
@pytest.mark.parametrize("with_entropy", [True, False])
def test_logits_gradients(dtype, rows, vocab, with_entropy):
    """Tolerances as for the small ones; a sum of a row passes vocab / 2048 + 40 additions in the forward kernel here
    (256 lanes at least, then 6 in a wave and 8 over the waves)."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    say("streamed logits", dtype, rows, vocab, with_entropy)
    x = (torch.randn(rows, vocab, generator=g, device=DEV) * 3).to(DT[dtype])
    tokens = torch.randint(0, vocab, (rows, 3), generator=g, device=DEV)
    tokens[:, 0] = x.float().argmax(1)
    tokens[::7, 2] = -1
    d_logp = torch.randn(rows, 3, generator=g, device=DEV)
    d_entropy = torch.randn(rows, generator=g, device=DEV) if with_entropy else None
    f = pc.pc_logprobs(x, tokens, scale=0.75)
    r = pc.pc_logprobs_backward(x, f.stats, tokens, d_logp, d_entropy, scale=0.75)
    for i in range(0, rows, 300):
        part = slice(i, i + 300)
        z = x[part].double() * 0.75
        top = z.amax(1, keepdim=True)
        log_s = (z - top).exp().sum(1, keepdim=True).log()
        y, logp = (z - top).abs(), z - top - log_s
        p = logp.exp()
        entropy = -(p * logp).sum(1, keepdim=True)
        d = torch.where(tokens[part] >= 0, d_logp[part].double(), 0.0)
        de = d_entropy[part].double()[:, None] if with_entropy else torch.zeros_like(entropy)
        at = tokens[part].clamp(min=0)
        onto = torch.zeros_like(p).scatter_add_(1, at, d)
        given = torch.zeros_like(p).scatter_add_(1, at, d.abs())
        want = 0.75 * (onto - p * (d.sum(1, keepdim=True) + de * (logp + entropy)))
        e = U * (vocab / 2048 + 46 + 4 * entropy) + 2 * U * log_s.abs()
        rel = e + 4 * U * (y + logp.abs()) + 4 * U * logp.abs() + 2 * U
        size = d.abs().sum(1, keepdim=True) + de.abs() * (logp.abs() + entropy)
        tol = 0.75 * (p * size * (rel + 15 * U) + p * de.abs() * ((3 * e + 20 * U) * (1 + entropy + log_s.abs()) + rel)
                      + 7 * U * (given + (given > 0) * p * size))
        check(r[part], want, tol, dtype)
        # the forward pass, bounded by the additions it has
        picked = torch.where(tokens[part] >= 0, logp.gather(1, at), 0.0)
        check(f.logp[part], picked, e + 4 * U * (y.gather(1, at) + picked.abs()), "f32")
        check(f.entropy[part], entropy[:, 0], ((3 * e + 20 * U) * (1 + entropy + log_s.abs()))[:, 0], "f32")
