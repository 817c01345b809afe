"""The stored-tensor and embedding operators on the GPU against their plain
64-bit forms (oracle/q8.py).

Tolerances, fixed before the first run:
* store: symbols and codes equal, byte for byte; load and lookup: the exact
  value (or the 32-bit product with the scale) rounded once: equal.
* activation backward: with w = exp(-|z|) from a 32-bit exponent and two
  reciprocals, the sigmoid is off by at most 5e-7 and its product with the
  polynomial's slope by 1e-6; the GELU tail adds 0.75e-7 (half of 7.1.26's
  bound).  So act is off by at most 1e-6 |g| and act' by 2e-6 (1 + |g| there is
  absorbed by the exponential), times the other factors, plus half a step of
  the output's type (a relative 2^-24, 2^-11 or 2^-8) and its smallest number.
* sums of m exact terms in 32 bits, in any order: at most (m + 2) 2^-23 times
  the sum of the terms' magnitudes (one bit more than rounding to nearest
  needs, as the matrix instructions do not say how they round), plus half a
  step of the output's type.
"""
import math
import sys

import numpy as np
import pytest
import torch

from oracle import q8

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}


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


def activation(rng, rows, cols, dtype):
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)))
    return tensor(x.astype(np.float32), dtype)


def make_q8(rng, rows, cols, fmt, scale=1.0):
    """A stored tensor straight from the oracle, and its values."""
    sym, codes = q8.store(rng.normal(size=(rows, cols)) * scale, fmt)
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), fmt)
    return q, q8.load(sym, codes, fmt)


def same(got, want):
    """Equal, NaN to NaN."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape
    ok = (got == want) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (int((~ok).sum()), got[~ok][:4], want[~ok][:4])


def within(got, want, tol):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape
    off = np.abs(got - want) - tol
    assert np.all(np.isfinite(got)) and np.all(off <= 0), (float(off.max()), int((off > 0).sum()))


def rounded(a, dtype):
    """64-bit numbers that 32 bits hold, rounded to the type."""
    return np64(torch.from_numpy(np.asarray(a, dtype=np.float64)).float().to(DT[dtype]))


# -- store and load ----------------------------------------------------------------

SIZES = [(1, 1), (1, 31), (1, 32), (2, 33), (3, 7), (5, 64), (7, 1000), (1, 4096), (33, 257), (130, 96), (2, 8191),
         (1023, 8)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_store_and_load(dtype, fmt):
    rng = np.random.default_rng(5)
    for rows, cols in SIZES:
        say("store", rows, cols, dtype, fmt)
        x = activation(rng, rows, cols, dtype)
        counts = torch.full((256,), 3, dtype=torch.int64, device=DEV)
        q = pc.pc_q8_store(x, fmt, counts=counts)
        plain = pc.pc_q8_store(x, fmt)
        sym, codes = q8.store(np64(x), fmt)
        for s in (q, plain):
            assert np.array_equal(s.symbols.cpu().numpy(), sym)
            assert np.array_equal(s.scales.cpu().numpy(), codes)
        assert np.array_equal(counts.cpu().numpy(), 3 + np.bincount(sym.reshape(-1), minlength=256))
        for to in ("f32", "f16", "bf16"):
            same(np64(pc.pc_q8_load(q, DT[to])), rounded(q8.load(sym, codes, fmt), to))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_at_the_edges_of_the_range(fmt):
    inf, nan = math.inf, math.nan
    rows = [
        [0.0] * 40,
        [-0.0] * 40,
        [nan] * 40,
        [inf, -inf] * 20,
        [1.0, nan, -inf, 2.0 ** -9] + [0.25] * 36,
        [2.0 ** -126, 2.0 ** -149] + [0.0] * 38,
        [2.0 ** -109] * 20 + [2.0 ** -120] * 20,
        [3.0e38, 1.0, -3.0e38] + [1e30] * 37,
        [448.0, 448.1, -447.9] + [0.5 * 2.0 ** -9] * 37,
        [127.0, 126.5, -0.5, 0.5, 1.5, 2.5] + [100.0] * 34,
        [float(np.nextafter(np.float32(448), np.float32(1e9)))] * 40,
        [1.75 * 2.0 ** k for k in range(-20, 20)],
    ]
    x = np.array(rows, dtype=np.float32)
    t = torch.from_numpy(x).to(DEV)
    q = pc.pc_q8_store(t, fmt)
    sym, codes = q8.store(x.astype(np.float64), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), codes)
    assert np.array_equal(q.symbols.cpu().numpy(), sym)
    back = np64(pc.pc_q8_load(q, torch.float32))
    assert np.array_equal(np.isnan(back), ~np.isfinite(x))
    same(back, rounded(q8.load(sym, codes, fmt), "f32"))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_load_every_symbol_and_code(fmt):
    sym = np.tile(np.arange(256, dtype=np.uint8), (254, 1))
    codes = np.repeat(np.arange(1, 255, dtype=np.uint8)[:, None], 8, axis=1)
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), fmt)
    want = q8.load(sym, codes, fmt)
    for to in ("f32", "bf16", "f16"):
        same(np64(pc.pc_q8_load(q, DT[to])), np64(torch.from_numpy(want).float().to(DT[to])))


def test_store_and_load_of_views():
    rng = np.random.default_rng(6)
    big = activation(rng, 20, 300, "bf16")
    for x in (big[2:9, 5:133], big[::3, :64], big.view(4, 5, 300)[1:3], big[3], big[4:5, 1:2]):
        q = pc.pc_q8_store(x, "e4m3")
        flat = np64(x).reshape(-1, x.shape[-1])
        sym, codes = q8.store(flat, "e4m3")
        assert np.array_equal(q.symbols.cpu().numpy(), sym) and np.array_equal(q.scales.cpu().numpy(), codes)
    out = torch.full((7, 200), -1.0, device=DEV)
    q, v = make_q8(rng, 7, 100, "int8")
    pc.pc_q8_load(q, torch.float32, out=out[:, 3:103])
    same(np64(out[:, 3:103]), v)
    assert torch.all(out[:, :3] == -1) and torch.all(out[:, 103:] == -1)
    part = q.columns(32, 96)
    same(np64(pc.pc_q8_load(part, torch.float32)), v[:, 32:96])
    with pytest.raises(ValueError):
        q.columns(8, 96)
    with pytest.raises(ValueError):
        pc.pc_q8_store(big.t())
    with pytest.raises(ValueError):
        pc.pc_q8_store(big.view(4, 5, 300).transpose(0, 1))
    with pytest.raises(TypeError):
        pc.pc_q8_load(q, torch.float64)
    with pytest.raises(TypeError):
        pc.pc_q8_load(q, torch.float16, out=out[:, :100])
    with pytest.raises(ValueError):
        pc.pc_q8_load(q, torch.float32, out=out)


def test_nothing_to_store():
    assert pc.pc_q8_store(torch.empty((2, 3, 0), device=DEV)).shape == (6, 0)
    for shape in ((0, 64), (5, 0), (0, 0)):
        q = pc.pc_q8_store(torch.empty(shape, device=DEV))
        assert q.symbols.shape == shape and pc.pc_q8_load(q).shape == shape


def test_offsets_past_32_bits():
    # a row distance that puts the second row 5 GB away, and tables of 5 GB
    rng = np.random.default_rng(7)
    ld = 5 * (1 << 29)
    buf = torch.zeros(ld + 1000, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((2, 1000), (ld, 1))
    x.copy_(activation(rng, 2, 1000, "bf16"))
    q = pc.pc_q8_store(x, "e4m3")
    sym, codes = q8.store(np64(x), "e4m3")
    assert np.array_equal(q.symbols.cpu().numpy(), sym) and np.array_equal(q.scales.cpu().numpy(), codes)
    back = torch.zeros(ld + 1000, dtype=torch.bfloat16, device=DEV).as_strided((2, 1000), (ld, 1))
    pc.pc_q8_load(q, torch.bfloat16, out=back)
    same(np64(back), q8.load(sym, codes, "e4m3"))
    del buf, x, back
    vocab, dim = 5_000_001, 1024
    table = torch.zeros((vocab, dim), dtype=torch.uint8, device=DEV)
    scales = torch.full((vocab, dim // 32), 127, dtype=torch.uint8, device=DEV)
    table[vocab - 1] = 0x38  # 1.0
    tokens = torch.tensor([vocab - 1, 0], device=DEV)
    out = pc.pc_embed(tokens, pc.Q8(table, scales, "e4m3"), scale=3.0)
    assert torch.all(out[0] == 3.0) and torch.all(out[1] == 0.0)
    del table, scales
    grad = torch.ones((3_000_001, 1024), dtype=torch.bfloat16, device=DEV)
    dy = torch.full((3, 1024), 0.5, dtype=torch.bfloat16, device=DEV)
    pc.pc_embed_backward(dy, torch.tensor([3_000_000, 5, 3_000_000], device=DEV), 3_000_001, dtype=torch.bfloat16,
                         out=grad)
    assert torch.all(grad[3_000_000] == 1.0) and torch.all(grad[5] == 0.5)
    assert torch.count_nonzero(grad).item() == 2048


# -- activation backward -------------------------------------------------------------

def check_glu(dh, g, u, act, dtype, grads, h=None):
    dg, du, hh = q8.glu_backward(dh, g, 1.0 if u is None else u, act)
    uu = np.abs(np.ones_like(g) if u is None else u)
    half, tiny = HALF_STEP[dtype], TINY[dtype]

    def bound(value, slack):
        return slack + half * (np.abs(value) + slack) + tiny + 4 * 2.0 ** -24 * np.abs(value)

    within(np64(grads.gate), dg, bound(dg, np.abs(dh) * uu * 2e-6))
    if u is not None:
        within(np64(grads.up), du, bound(du, np.abs(dh * g) * 1e-6))
    if h is not None:
        within(np64(h), hh, bound(hh, np.abs(g) * uu * 1e-6))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_glu_backward(dtype, fmt, act):
    rng = np.random.default_rng(8)
    for rows, cols in [(1, 1), (3, 32), (2, 45), (9, 128), (4, 1000), (65, 96)]:
        say("glu", rows, cols, dtype, fmt, act)
        gate, g = make_q8(rng, rows, cols, fmt, 3.0)
        up, u = make_q8(rng, rows, cols, fmt)
        dh = tensor(rng.normal(size=(rows, cols)).astype(np.float32), dtype)
        r = pc.pc_q8_glu_backward(dh, gate, up, act=act, with_h=True)
        check_glu(np64(dh), g, u, act, dtype, r, r.h)
        r = pc.pc_q8_glu_backward(dh, gate, up, act=act)
        assert r.h is None
        check_glu(np64(dh), g, u, act, dtype, r)
        r = pc.pc_q8_glu_backward(dh, gate, act=act, with_h=True)
        assert r.up is None
        check_glu(np64(dh), g, None, act, dtype, r, r.h)
        if cols % 32 == 0:
            both = pc.Q8(torch.cat([gate.symbols, up.symbols], 1), torch.cat([gate.scales, up.scales], 1), fmt)
            r = pc.pc_q8_glu_backward(dh, both, act=act, with_h=True)
            assert r.packed.shape == (rows, 2 * cols)
            check_glu(np64(dh), g, u, act, dtype, r, r.h)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_glu_backward_far_out_and_nan(act):
    # values at which the exponential over- and underflows: the ends of every form
    sym = np.tile(np.array([0x7E, 0xFE, 0x7F, 0x00, 0x80, 0x38, 0xB8, 0x48], dtype=np.uint8), (6, 4))
    codes = np.array([[127], [120], [130], [150], [190], [210]], dtype=np.uint8)
    q = pc.Q8(torch.from_numpy(sym).to(DEV), torch.from_numpy(codes).to(DEV), "e4m3")
    v = q8.load(sym, codes, "e4m3")
    dh = torch.ones(6, 32, device=DEV)
    r = pc.pc_q8_glu_backward(dh, q, act=act, with_h=True)
    for got, f in ((r.gate, q8.act_slope), (r.h, q8.act)):
        got = np64(got)
        for i in np.ndindex(*v.shape):
            g = v[i]
            if math.isnan(g):
                assert math.isnan(got[i])
                continue
            if abs(g) > 50:  # the identity, or nothing
                want = (1.0 if f is q8.act_slope else g) if g > 0 else 0.0
            else:
                want = float(f(act, np.array(g)))
            assert abs(got[i] - want) <= 2e-6 * max(1.0, abs(want)), (g, got[i], want)


def test_glu_backward_is_the_slope_of_the_forward_pass():
    rng = np.random.default_rng(9)
    gate, g = make_q8(rng, 3, 64, "int8", 2.0)
    up, u = make_q8(rng, 3, 64, "int8")
    dh = rng.normal(size=(3, 64)).astype(np.float32)
    for act in ("silu", "gelu", "gelu_tanh"):
        r = pc.pc_q8_glu_backward(tensor(dh, "f32"), gate, up, act=act)
        e = 1e-4
        dg = dh * u * (q8.act(act, g + e) - q8.act(act, g - e)) / (2 * e)
        du = dh * q8.act(act, g) * ((u + e) - (u - e)) / (2 * e)
        # differences of a smooth function: e^2 / 6 of a third derivative below 3
        assert np.max(np.abs(np64(r.gate) - dg)) < 1e-5 and np.max(np.abs(np64(r.up) - du)) < 2e-5


def test_glu_backward_in_place_and_of_views():
    rng = np.random.default_rng(10)
    gate, g = make_q8(rng, 5, 96, "e4m3", 2.0)
    up, u = make_q8(rng, 5, 96, "e4m3")
    wide = tensor(rng.normal(size=(5, 300)).astype(np.float32), "bf16")
    dh = wide[:, 7:103]
    check_glu(np64(dh), g, u, "silu", "bf16", pc.pc_q8_glu_backward(dh, gate, up))
    d = dh.contiguous()
    want = pc.pc_q8_glu_backward(d, gate, up).gate.clone()
    lib = pc._lib.lib
    du = torch.empty_like(d)
    st = lib.pc_q8_glu_backward(d.data_ptr(), 2, 96, gate.arg, up.arg, 0, d.data_ptr(), 96, du.data_ptr(), 96, None, 0,
                                torch.cuda.current_stream().cuda_stream)
    assert st == pc.PC_OK and torch.equal(d, want)
    with pytest.raises(ValueError):
        pc.pc_q8_glu_backward(dh[:, :95], gate, up)
    with pytest.raises(ValueError):
        pc.pc_q8_glu_backward(dh[:, :50], gate)
    with pytest.raises(ValueError):
        pc.pc_q8_glu_backward(dh, gate, act="relu")
    odd, _ = make_q8(rng, 5, 90, "e4m3")
    with pytest.raises(ValueError):
        pc.pc_q8_glu_backward(dh[:, :45], odd)  # gate and up would share a group


# -- weight gradient -----------------------------------------------------------------

def check_wgrad(dy, x, got, odt, old=None):
    want = q8.weight_grad(dy, x)
    size = np.abs(dy).T @ np.abs(x)
    if old is not None:
        want, size = want + old, size + np.abs(old)
    within(np64(got), want, (dy.shape[0] + 3) * 2.0 ** -23 * size + HALF_STEP[odt] * np.abs(want) + TINY[odt])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight_grad(dtype, fmt):
    rng = np.random.default_rng(11)
    for t, n, k, odt in [(1, 1, 1, "f32"), (1, 40, 33, "bf16"), (7, 9, 100, "f32"), (64, 128, 128, "f32"),
                         (65, 129, 127, "f16"), (200, 257, 300, "f32"), (1000, 64, 96, "bf16"), (3001, 31, 65, "f32"),
                         (300, 520, 264, "f32")]:
        say("wgrad", t, n, k, dtype, fmt, odt)
        q, x = make_q8(rng, t, k, fmt)
        dy = activation(rng, t, n, dtype)
        check_wgrad(np64(dy), x, pc.pc_q8_weight_grad(dy, q, dtype=DT[odt]), odt)
        old = tensor(rng.normal(size=(n, k)).astype(np.float32), odt)
        out = old.clone()
        pc.pc_q8_weight_grad(dy, q, dtype=DT[odt], out=out, accumulate=True)
        check_wgrad(np64(dy), x, out, odt, np64(old))


@pytest.mark.parametrize("t,n,k,fmt", [(777, 4200, 3976, "e4m3"), (640, 4096, 3840, "e4m3"), (333, 4096, 3840, "int8"),
                                       (200, 4099, 3845, "int8"), (70, 4099, 3845, "e4m3")])
def test_weight_grad_of_many_tiles(t, n, k, fmt):
    # the large tiles, whole and ragged on every side; products against 64-bit ones on the device
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(t, k, generator=g, device=DEV)
    dy = torch.randn(t, n, generator=g, device=DEV).to(torch.bfloat16)
    q = pc.pc_q8_store(x, fmt)
    v = pc.pc_q8_load(q, torch.float32).double()
    want = torch.mm(dy.double().t().contiguous(), v)
    size = torch.mm(dy.double().abs().t().contiguous(), v.abs())
    got = pc.pc_q8_weight_grad(dy, q)
    tol = (t + 3) * 2.0 ** -23 * size + 2.0 ** -24 * want.abs()
    assert bool((torch.abs(got.double() - want) <= tol).all())
    half = pc.pc_q8_weight_grad(dy, q, dtype=torch.bfloat16)
    assert bool((torch.abs(half.double() - want) <= tol + 2.0 ** -8 * want.abs()).all())
    pc.pc_q8_weight_grad(dy, q, out=got, accumulate=True)
    assert bool((torch.abs(got.double() - 2 * want) <= 3 * tol).all())


def test_weight_grad_of_views_and_nothing():
    rng = np.random.default_rng(12)
    q, x = make_q8(rng, 90, 128, "int8")
    wide = activation(rng, 90, 200, "bf16")
    dy = wide[:, 3:78]
    out = torch.full((75, 150), 7.0, device=DEV)
    pc.pc_q8_weight_grad(dy, q.columns(32, 96), out=out[:, 5:69])
    check_wgrad(np64(dy), x[:, 32:96], out[:, 5:69], "f32")
    assert torch.all(out[:, :5] == 7) and torch.all(out[:, 69:] == 7)
    nothing = pc.Q8(torch.empty((0, 40), dtype=torch.uint8, device=DEV),
                    torch.empty((0, 2), dtype=torch.uint8, device=DEV))
    none = torch.empty((0, 8), dtype=torch.bfloat16, device=DEV)
    assert torch.all(pc.pc_q8_weight_grad(none, nothing) == 0)
    keep = torch.full((8, 40), 2.0, device=DEV)
    pc.pc_q8_weight_grad(none, nothing, out=keep, accumulate=True)
    assert torch.all(keep == 2.0)
    pc.pc_q8_weight_grad(none, nothing, out=keep)
    assert torch.all(keep == 0.0)
    assert pc.pc_q8_weight_grad(dy[:, :0], q).shape == (0, 128)
    with pytest.raises(ValueError):
        pc.pc_q8_weight_grad(dy[:50], q)
    with pytest.raises(ValueError):
        pc.pc_q8_weight_grad(dy, q, accumulate=True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight_grad_carries_infinity_and_nan(dtype, fmt):
    rng = np.random.default_rng(13)
    q, x = make_q8(rng, 40, 64, fmt)
    dy = np.ones((40, 16), dtype=np.float32)
    dy[3, 2], dy[5, 4] = math.inf, math.nan
    sym = q.symbols.clone()
    sym[7, 9] = q8.NAN_BYTE[fmt]
    got = np64(pc.pc_q8_weight_grad(tensor(dy, dtype), q.with_symbols(sym)))
    v = x.copy()
    v[7, 9] = math.nan
    with np.errstate(invalid="ignore"):
        want = dy.astype(np.float64).T @ v
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    assert np.max(np.abs(got[fine] - want[fine])) < 1e-3


def test_weight_grad_is_the_same_every_time():
    rng = np.random.default_rng(14)
    q, _ = make_q8(rng, 5000, 96, "e4m3")
    dy = activation(rng, 5000, 40, "bf16")
    first = pc.pc_q8_weight_grad(dy, q)
    for _ in range(5):
        assert torch.equal(first, pc.pc_q8_weight_grad(dy, q))


# -- embedding -----------------------------------------------------------------------

@pytest.mark.parametrize("table", ["f32", "f16", "bf16", "e4m3", "int8"])
def test_embed(table):
    rng = np.random.default_rng(15)
    for vocab, dim, shape in [(1, 1, (1,)), (10, 33, (3, 5)), (100, 256, (70,)), (50, 1000, (2, 1, 9)), (7, 40, ())]:
        if table in DT:
            tab = tensor(rng.normal(size=(vocab, dim)).astype(np.float32), table)
            v = np64(tab)
        else:
            tab, v = make_q8(rng, vocab, dim, table)
        tokens = rng.integers(0, vocab, shape)
        scale = math.sqrt(dim)
        # one product in 32 bits
        want32 = (v.astype(np.float32)[tokens] * np.float32(scale)).astype(np.float64)
        for ity in (torch.int64, torch.int32):
            for out in ("f32", "f16", "bf16"):
                say("embed", vocab, dim, shape, table, out)
                got = pc.pc_embed(torch.from_numpy(np.array(tokens)).to(ity).to(DEV), tab, scale=scale, dtype=DT[out])
                assert got.shape == (*shape, dim)
                same(np64(got), rounded(want32, out))


def test_embed_outside_the_table():
    table = torch.ones(6, 50, device=DEV)
    tokens = torch.tensor([0, -1, 6, 5, 1 << 40, -(1 << 40)], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pc.pc_embed(tokens, table, status=status)
    assert int(status.item()) == pc.PC_ERR_INVALID_ARG
    assert out.sum(1).tolist() == [50, 0, 0, 50, 0, 0]
    status.zero_()
    pc.pc_embed(tokens[3:4], table, status=status)
    assert int(status.item()) == 0
    assert torch.all(pc.pc_embed(tokens[:4], table[:0]) == 0)
    assert pc.pc_embed(tokens[:0], table).shape == (0, 50)
    wide = torch.full((3, 80), 9.0, device=DEV)
    pc.pc_embed(torch.tensor([1, 2, 3], device=DEV), table[:, 4:44], out=wide[:, 8:48])
    assert torch.all(wide[:, 8:48] == 1) and torch.all(wide[:, :8] == 9) and torch.all(wide[:, 48:] == 9)
    with pytest.raises(TypeError):
        pc.pc_embed(tokens.float(), table)
    with pytest.raises(ValueError):
        pc.pc_embed(tokens, table, out=wide)


def token_cases(rng, n, vocab):
    yield "spread", rng.integers(0, vocab, n)
    yield "one", np.full(n, vocab // 2)
    yield "few", rng.integers(0, min(vocab, 3), n)
    yield "ends", np.where(rng.random(n) < 0.5, 0, vocab - 1)
    yield "skewed", np.minimum((vocab * rng.random(n) ** 6).astype(np.int64), vocab - 1)
    bad = rng.integers(-3, vocab + 3, n)
    bad[rng.random(n) < 0.1] = 1 << 40
    yield "outside", bad


@pytest.mark.parametrize("dtype,odt", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("bf16", "f16")])
def test_embed_backward(dtype, odt):
    rng = np.random.default_rng(16)
    for n, dim, vocab in [(1, 1, 1), (1, 64, 9), (31, 33, 50), (32, 520, 7), (33, 8, 300), (500, 40, 70),
                          (1000, 17, 3000), (3000, 24, 257)]:
        for name, tokens in token_cases(rng, n, vocab):
            say("embed backward", n, dim, vocab, dtype, odt, name)
            dy = activation(rng, n, dim, dtype)
            t = torch.from_numpy(tokens).to(DEV)
            padding = 1 if name == "few" else -1
            want, size, terms = q8.embed_backward(np64(dy), tokens, vocab, 0.37, padding)
            tol = (terms[:, None] + 3) * 2.0 ** -23 * size + HALF_STEP[odt] * np.abs(want) + TINY[odt] * (size > 0)
            got = pc.pc_embed_backward(dy, t, vocab, scale=0.37, dtype=DT[odt], padding=padding)
            within(np64(got), want, tol)
            assert torch.equal(got, pc.pc_embed_backward(dy, t, vocab, scale=0.37, dtype=DT[odt], padding=padding))
            if name != "outside":
                assert torch.equal(got, pc.pc_embed_backward(dy, t.int(), vocab, scale=0.37, dtype=DT[odt],
                                                             padding=padding))
            old = tensor(rng.normal(size=(vocab, dim)).astype(np.float32), odt)
            out = old.clone()
            pc.pc_embed_backward(dy, t, vocab, scale=0.37, dtype=DT[odt], padding=padding, out=out, accumulate=True)
            o = np64(old)
            within(np64(out), want + o, tol + (np.abs(o) * 2.0 ** -23 + HALF_STEP[odt] * np.abs(want + o)) * (size > 0))


def test_embed_backward_larger():
    # vocabularies of several ranges, more tokens than one pass of a workgroup, on the device in 64 bits
    g = torch.Generator(device=DEV).manual_seed(3)
    for n, dim, vocab, skew in [(1024, 520, 200000, 1), (1025, 520, 9000, 6), (5000, 96, 20000, 1), (40000, 64, 50257, 6), (20000, 40, 300000, 3),
                                (70000, 16, 1000, 1)]:
        say("embed backward", n, dim, vocab)
        u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
        tokens = (u ** skew * vocab).long().clamp_(max=vocab - 1)
        dy = torch.randn(n, dim, generator=g, device=DEV).to(torch.bfloat16)
        got = pc.pc_embed_backward(dy, tokens, vocab)
        want = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV).index_add_(0, tokens, dy.double())
        size = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV).index_add_(0, tokens, dy.double().abs())
        terms = torch.bincount(tokens, minlength=vocab).unsqueeze(1)
        assert bool((torch.abs(got.double() - want) <= (terms + 3) * 2.0 ** -23 * size).all())
        assert torch.equal(got, pc.pc_embed_backward(dy, tokens, vocab))
        pc.pc_embed_backward(dy, tokens, vocab, out=got, accumulate=True)
        assert bool((torch.abs(got.double() - 2 * want) <= (2 * terms + 6) * 2.0 ** -23 * size).all())


def test_embed_backward_of_nothing_and_views():
    none = torch.empty(0, 12, device=DEV)
    no_tokens = torch.empty(0, dtype=torch.int64, device=DEV)
    assert torch.all(pc.pc_embed_backward(none, no_tokens, 5) == 0)
    keep = torch.full((5, 12), 3.0, device=DEV)
    pc.pc_embed_backward(none, no_tokens, 5, out=keep, accumulate=True)
    assert torch.all(keep == 3)
    wide = torch.ones(6, 40, device=DEV)
    out = torch.full((4, 30), -1.0, device=DEV)
    pc.pc_embed_backward(wide[::2, 3:15], torch.tensor([2, 0, 2], device=DEV), 4, out=out[:, 9:21])
    assert out[:, 9:21].sum(1).tolist() == [12, 0, 24, 0]
    assert torch.all(out[:, :9] == -1) and torch.all(out[:, 21:] == -1)
    with pytest.raises(ValueError):
        pc.pc_embed_backward(wide, torch.tensor([2, 0], device=DEV), 4)
    with pytest.raises(ValueError):
        pc.pc_embed_backward(wide[:2], torch.tensor([2, 0], device=DEV), 4, accumulate=True)


# -- streams and graphs --------------------------------------------------------------

def all_operators(x, dh, q, tokens, table):
    counts = torch.zeros(256, dtype=torch.int64, device=DEV)
    s = pc.pc_q8_store(x, "e4m3", counts=counts)
    r = pc.pc_q8_glu_backward(dh, s, act="gelu", with_h=True)
    dw = pc.pc_q8_weight_grad(r.gate, q)
    e = pc.pc_embed(tokens, table, scale=2.0)
    de = pc.pc_embed_backward(e, tokens, table.shape[0])
    return [s.symbols, s.scales, counts, pc.pc_q8_load(s), r.gate, r.h, dw, e, de]


def operator_inputs(seed):
    rng = np.random.default_rng(seed)
    x, dh = activation(rng, 600, 96, "bf16"), activation(rng, 600, 96, "bf16")
    q, _ = make_q8(rng, 600, 70, "e4m3")
    return x, dh, q, torch.from_numpy(rng.integers(0, 50, 600)).to(DEV), activation(rng, 50, 128, "bf16")


def test_on_another_stream():
    args = operator_inputs(17)
    want = all_operators(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_operators(*args)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_in_a_graph():
    args = operator_inputs(18)
    all_operators(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_operators(*args)
    for seed in (19, 20, 21):
        fresh = operator_inputs(seed)
        for a, b in zip(args, fresh):
            if isinstance(a, torch.Tensor):
                a.copy_(b)
            else:
                a.symbols.copy_(b.symbols)
                a.scales.copy_(b.scales)
        want = all_operators(*fresh)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# -- with the coder --------------------------------------------------------------------

def test_stored_symbols_through_the_coder():
    rng = np.random.default_rng(22)
    x = activation(rng, 64, 512, "bf16")
    counts = torch.zeros(256, dtype=torch.int64, device=DEV)
    q = pc.pc_q8_store(x, "e4m3", counts=counts)
    assert torch.equal(counts, pc.pc_histogram(q.symbols))
    book = pc.pc_codebook_build(counts).to(DEV)
    enc = pc.pc_encode(book, q.symbols, 4096)
    back, status = pc.pc_decode(book, enc)
    assert int(status.item()) == 0
    again = q.with_symbols(back)
    assert torch.equal(again.symbols, q.symbols)
    assert torch.equal(pc.pc_q8_load(again), pc.pc_q8_load(q))
