"""The norm where a product of two of its factors leaves the range of 32 bits,
and where its output comes to the end of it.  Tolerances are those of
test_gpu_step.py: y has 3.1 u, and the stored form equals that of y in 64 bits,
byte for byte."""
import numpy as np
import pytest
import torch

from oracle import q8, step
from test_gpu_step import DEV, DT, EPS, U, check_stored, np64, say, tensor, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def faint_row(rng, cols):
    """(h, weight): of each 32 columns, some that make the row's size, and some that are small beside it but for their weights."""
    h, w = rng.normal(size=cols), 0.5 + rng.random(cols)
    kind = np.arange(cols) // 32 % 5
    h[kind == 0] *= 1e19
    for k, size, weight in ((1, 1e-26, 1e10),    # h rstd of some 1e-45: few digits in 32 bits
                            (2, 1e-31, 1e30),    # none
                            (3, 3e-39, 1e25),    # from an h below the normal range
                            (4, 1e-20, 1e3)):    # of some 1e-39
        h[kind == k] *= size
        w[kind == k] *= weight
    return h, w


@pytest.mark.parametrize("dtype,res", [("f32", None), ("bf16", None), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_small_numbers_with_large_weights(dtype, res, fmt):
    rng = np.random.default_rng(61)
    for cols in (128, 250, 256, 640, 4104, 8192, 16390, 16400, 33000):
        say("faint", cols, dtype, res, fmt)
        rows = [faint_row(rng, cols)[0] for _ in range(2)] + [rng.normal(size=cols)]
        w = tensor(faint_row(rng, cols)[1].astype(np.float32), "f32")
        h = np.stack(rows).astype(np.float32)
        if res is None:
            x, residual = tensor(h, dtype), None
        else:
            x, residual = torch.zeros(3, cols, dtype=DT[dtype], device=DEV), tensor(h, res)
        r = pc.pc_rmsnorm_store(x, w, residual, format=fmt, y="plain", dtype=torch.float32)
        y, _ = step.norm(np64(r.sum), np64(w), EPS)
        within(np64(r.y), y, 3.1 * U * np.abs(y))
        check_stored(r.q, y, fmt)
        counts = torch.zeros(256, dtype=torch.int64, device=DEV)
        c = pc.pc_rmsnorm_store(x, w, residual, format=fmt, counts=counts, y="stored", dtype=torch.float32)
        assert torch.equal(c.q.symbols, r.q.symbols) and torch.equal(c.q.scales, r.q.scales)
        assert np.array_equal(np64(c.y), q8.load(r.q.symbols.cpu().numpy(), r.q.scales.cpu().numpy(), fmt))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_reciprocal_roots_below_the_normal_range(dtype):
    """Rows of a size above 2^126, whose reciprocal keeps fewer digits in 32 bits than y has."""
    rng = np.random.default_rng(62)
    for cols in (64, 250, 2048, 16400, 33000):
        say("large rows", cols, dtype)
        x = tensor((rng.uniform(0.5, 1, size=(4, cols)) * rng.choice([-1, 1], size=(4, cols)) * 3.3e38).astype(np.float32), dtype)
        w = tensor((1 + 0.3 * rng.normal(size=cols)).astype(np.float32), "f32")
        for fmt in ("e4m3", "int8"):
            r = pc.pc_rmsnorm_store(x, w, format=fmt, y="plain", dtype=torch.float32)
            y, _ = step.norm(np64(x), np64(w), EPS)
            within(np64(r.y), y, 3.1 * U * np.abs(y))
            check_stored(r.q, y, fmt)


END = 2.0 ** 128 - 2.0 ** 103  # from here on 32 bits round to infinity


def ends():
    """(h, weight) of which y in 64 bits rounds to the largest number of 32 bits, and products in 32 bits to infinity, and the reverse."""
    found = {}
    for h in 1 + np.arange(1, 40, dtype=np.float32) / 64:
        rstd = 1 / np.sqrt(np.float64(h) ** 2 / 64 + EPS)
        first = np.float32(END / (np.float64(h) * rstd))
        for k in range(-4, 5):
            w = np.float32(first + k * np.spacing(first))
            exact = np.float64(h) * rstd * np.float64(w)
            with np.errstate(over="ignore"):
                product = np.float32(np.float32(h * np.float32(rstd)) * w)
            if np.isinf(product) != (exact >= END):
                found[bool(exact >= END)] = h, w
    return found


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_stored_outputs_at_the_end_of_the_range(dtype):
    found = ends()
    assert set(found) == {False, True}
    for h, w in found.values():
        x, weight = torch.zeros(2, 64, device=DEV), torch.ones(64, device=DEV)
        x[:, 0], weight[0] = float(h), float(w)
        x = x.to(DT[dtype])
        for fmt in ("e4m3", "int8"):
            r = pc.pc_rmsnorm_store(x, weight, format=fmt)
            y, _ = step.norm(np64(x), np64(weight), EPS)
            check_stored(r.q, np.where(y >= END, np.inf, y), fmt)
