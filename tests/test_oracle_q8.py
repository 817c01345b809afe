"""The plain 64-bit forms of the stored-tensor operators, pinned on the CPU:
to the number format (torch's float8_e4m3fn), to closed forms, and the
gradients to central differences."""
import math

import numpy as np
import pytest
import torch

from oracle import q8


def test_elements_are_e4m3fn():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = q8.elements("e4m3")
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    assert max(v for v in got if not math.isnan(v)) == 448.0


def test_nearest_is_the_cast():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(0, 100, 400), rng.normal(0, 0.01, 400),
                        [0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, -(2.0 ** -10), 17.0, 19.0, 240.0]])
    y = np.clip(y, -448, 448).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [q8.nearest_byte(float(v), "e4m3") for v in y] == list(want)
    z = np.array([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5, 127.0, 3.2], dtype=np.float64)
    assert [q8.nearest_byte(float(v), "int8") for v in z] == [int(v) & 0xFF for v in np.rint(z)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_that_holds(fmt):
    for top in (1.0, 448.0, 448.0000001, 127.0, 127.00001, 255.9, 256.0, 3e38, 1e-30, 2.0 ** -126, 0.0):
        k = q8.exponent_for(top, fmt)
        assert top <= q8.MOST[fmt] * 2.0 ** k
        assert k == -117 or top > q8.MOST[fmt] * 2.0 ** (k - 1)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_array_forms_are_the_single_ones(fmt):
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.normal(0, 30, 300), q8.elements("e4m3")[:0x7F], -q8.elements("e4m3")[:0x7F],
                        (q8.elements("e4m3")[1:0x7F] + q8.elements("e4m3")[:0x7E]) / 2])
    y = np.clip(y, -q8.MOST[fmt], q8.MOST[fmt])
    assert list(q8.nearest_bytes(y, fmt)) == [q8.nearest_byte(float(v), fmt) for v in y]
    tops = np.concatenate([np.exp2(rng.uniform(-140, 127, 200)), [0.0, 1.0, 448.0, 127.0, 3.4e38]])
    assert [q8.exponent_near(float(v), fmt) for v in tops] == [q8.exponent_for(float(v), fmt) for v in tops]


@pytest.mark.parametrize("fmt,rel", [("e4m3", 2.0 ** -4), ("int8", 0.5)])
def test_round_trip_error(fmt, rel):
    x = np.random.default_rng(1).normal(0, 3, (5, 77))
    sym, codes = q8.store(x, fmt)
    back = q8.load(sym, codes, fmt)
    k = np.repeat(codes.astype(int) - 127, 32, axis=1)[:, :77]
    if fmt == "int8":
        assert np.all(np.abs(back - x) <= rel * np.exp2(k))
    else:  # half a step: 2^-4 of the number, or 2^-10 scaled among the smallest
        assert np.all(np.abs(back - x) <= np.maximum(rel * np.abs(x), 2.0 ** -10 * np.exp2(k)))
    again = q8.store(back, fmt)
    assert np.array_equal(q8.load(*again, fmt), back)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slopes_are_differences(name):
    g = np.linspace(-9, 9, 181)
    h = 1e-5
    diff = (q8.act(name, g + h) - q8.act(name, g - h)) / (2 * h)
    assert np.max(np.abs(diff - q8.act_slope(name, g))) < 1e-9


def test_linear_gradients_are_differences():
    rng = np.random.default_rng(2)
    dy, x, w = rng.normal(size=(7, 3)), rng.normal(size=(7, 4)), rng.normal(size=(3, 4))
    grad = q8.weight_grad(dy, x)
    for n in range(3):
        for k in range(4):
            e = np.zeros_like(w)
            e[n, k] = 0.5
            diff = np.sum(dy * (x @ (w + e).T)) - np.sum(dy * (x @ (w - e).T))
            assert abs(diff - grad[n, k]) < 1e-12
    tokens, table, up = np.array([2, 0, 2, 5, -1]), rng.normal(size=(4, 3)), rng.normal(size=(5, 3))
    grad, _, terms = q8.embed_backward(up, tokens, 4, 2.0)
    assert list(terms) == [1, 0, 2, 0]
    for v in range(4):
        for c in range(3):
            e = np.zeros_like(table)
            e[v, c] = 0.5
            diff = np.sum(up * q8.embed(tokens, table + e, 2.0)) - np.sum(up * q8.embed(tokens, table - e, 2.0))
            assert abs(diff - grad[v, c]) < 1e-12
