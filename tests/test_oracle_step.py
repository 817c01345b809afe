"""The plain 64-bit forms of the norm, dropout and log-probability operators:
against published values, differences, and torch's own operators."""
import math

import numpy as np
import pytest
import torch

from oracle import step


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD))])
def test_philox_known_answers(counter, key, want):
    """Known answers of Philox4x32-10 that its authors publish beside the paper."""
    assert tuple(step.philox(counter, key)) == want


def test_numbers_are_the_words_halves():
    n = step.numbers(3, 21, (7 << 32) | 5, (9 << 32) | 11)
    assert n.shape == (3, 21)
    for r in range(3):
        for c in range(21):
            w = step.philox((c // 8, r, 11, 9), (5, 7))[(c % 8) // 2]
            assert n[r, c] == (w >> 16 if c % 2 else w & 0xFFFF)


def test_dropout_keeps_the_mean():
    x = np.ones((400, 500))
    for p in (0.1, 0.5, 0.9):
        y = step.dropout(x, p, 3, 4)
        kept = 1 - step.below(p) / 65536
        assert np.allclose(y[y != 0], 1 / kept)
        # a binomial share of 200000: 5 standard deviations
        assert abs((y != 0).mean() - kept) < 5 * math.sqrt(kept * (1 - kept) / x.size)
    assert not step.dropout(x, 1.0, 3, 4).any() and np.array_equal(step.dropout(x, 0.0, 3, 4), x)
    gone = step.dropout(np.full((4, 64), np.nan), 0.5, 1, 2)
    assert np.isnan(gone).any() and (gone == 0).any()


def differences(f, x, d=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += d
        b[i] -= d
        g[i] = (f(a) - f(b)) / (2 * d)
    return g


def test_norm_backward_is_the_gradient():
    rng = np.random.default_rng(1)
    h, w, dy, ds = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    eps = 0.1
    got, dw = step.norm_backward(dy, h, w, step.rstd(h, eps), ds)

    def loss(h, w):
        return (step.norm(h, w, eps)[0] * dy).sum() + (h * ds).sum()
    # central differences: a third derivative of order 1 times d^2, and 1e-16 / d
    assert np.allclose(got, differences(lambda v: loss(v, w), h), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: loss(h, v), w), atol=1e-8)


def test_logprobs_against_torch():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(5, 40)) * 4
    x[1, 7:] = -np.inf
    x[2] = 3.0
    tokens = rng.integers(0, 7, size=(5, 3))
    tokens[0] = [-1, 40, -7]
    got, entropy, index, top = step.logprobs(x, tokens, 0.7, 6)
    want = torch.log_softmax(torch.from_numpy(x) * 0.7, 1)
    assert np.allclose(got[1:], want.gather(1, torch.from_numpy(tokens).clamp(0, 39)).numpy()[1:])
    assert (got[0] == 0).all()
    assert np.allclose(entropy, torch.special.entr(want.exp()).sum(1).numpy())
    assert np.array_equal(index[2], np.arange(6))  # all equal: by index
    assert np.array_equal(index[1], np.argsort(-x[1], kind="stable")[:6])
    assert np.allclose(top, np.take_along_axis(want.numpy(), index, 1))


def test_rows_that_leave_nothing():
    x = np.full((1, 9), -np.inf)
    got, entropy, index, top = step.logprobs(x, np.array([[0, 8]]), 1.0, 3)
    assert np.isneginf(got).all() and entropy[0] == 0 and np.array_equal(index, [[0, 1, 2]]) and np.isneginf(top).all()
    assert not step.logprobs_backward(x, np.array([[0, 8]]), 1.0, np.ones((1, 2)), np.ones(1)).any()


def test_logprobs_backward_is_the_gradient():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(3, 11))
    tokens = np.array([[1, 1, 4], [0, -1, 10], [2, 3, 99]])
    d, de = rng.normal(size=(3, 3)), rng.normal(size=3)

    def loss(x):
        logp, entropy, _, _ = step.logprobs(x, tokens, 1.3, 0)
        return (logp * d).sum() + (entropy * de).sum()
    assert np.allclose(step.logprobs_backward(x, tokens, 1.3, d, de), differences(loss, x), atol=1e-8)
