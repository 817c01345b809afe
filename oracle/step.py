"""Plain 64-bit forms of the norm, dropout and log-probability operators (numpy).

Written from the definitions in include/pc.h; shares no code or tables with the
library.
"""
from __future__ import annotations

import numpy as np

WORD = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10 of one counter (four words) and key (two words), in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & WORD, (a >> 32) ^ c[3] ^ k[1], a & WORD]
        k = [(k[0] + 0x9E3779B9) & WORD, (k[1] + 0xBB67AE85) & WORD]
    return c


def numbers(rows, cols, seed, offset):
    """The 16 bits of every element, by arrays of unsigned 64-bit words."""
    blocks = -(-cols // 8)
    u = np.uint64
    c = [np.tile(np.arange(blocks, dtype=u), rows), np.repeat(np.arange(rows, dtype=u), blocks),
         np.full(rows * blocks, offset & WORD, dtype=u), np.full(rows * blocks, offset >> 32, dtype=u)]
    k = [seed & WORD, seed >> 32]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & u(WORD), (a >> u(32)) ^ c[3] ^ u(k[1]), a & u(WORD)]
        k = [(k[0] + 0x9E3779B9) & WORD, (k[1] + 0xBB67AE85) & WORD]
    halves = [h for w in c for h in (w & u(0xFFFF), w >> u(16))]
    return np.stack(halves, 1).reshape(rows, blocks * 8)[:, :cols]


def below(p):
    return round(p * 65536)


def dropout(x, p, seed, offset):
    """mask(x): what is dropped is 0 whatever it held."""
    t = below(p)
    gone = numbers(*x.shape, seed, offset) < t
    with np.errstate(invalid="ignore"):
        return np.where(gone, 0.0, x * (65536 / (65536 - t) if t < 65536 else 0.0))


def rstd(h, eps):
    with np.errstate(over="ignore", invalid="ignore"):
        return 1 / np.sqrt((h * h).mean(1) + eps)


def norm(h, weight, eps):
    """(h rstd weight, rstd)"""
    r = rstd(h, eps)
    with np.errstate(invalid="ignore"):
        return h * r[:, None] * weight, r


def norm_backward(dy, h, weight, r, d_sum):
    """(d, d_weight) by the norm's Jacobian, r (I - n n^T / cols) with n = h r."""
    n = h * r[:, None]
    g = dy * weight
    d = r[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return d + d_sum, (dy * n).sum(0)


def log_softmax(x, scale):
    """log softmax(scale x) by rows; a row of -infinity gives -infinity throughout."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = x.max(1, keepdims=True)
        z = (x - np.where(np.isneginf(top), 0.0, top)) * scale
        logp = z - np.log(np.exp(z).sum(1, keepdims=True))
    return np.where(np.isneginf(top), -np.inf, logp)


def logprobs(x, tokens, scale, top, padding=-1):
    """(logp [rows, m], entropy, top indices, top logp)"""
    rows, vocab = x.shape
    logp = log_softmax(x, scale)
    p = np.exp(logp)
    with np.errstate(invalid="ignore"):
        entropy = -np.where(p == 0, 0.0, p * logp).sum(1)
    picked = np.zeros(tokens.shape)
    for r in range(rows):
        for j, t in enumerate(tokens[r]):
            if t != padding and 0 <= t < vocab:
                picked[r, j] = logp[r, t]
    key = np.where(np.isnan(x), -np.inf, x)
    index = np.argsort(-key, axis=1, kind="stable")[:, :top]
    return picked, entropy, index, np.take_along_axis(logp, index, 1)


def logprobs_backward(x, tokens, scale, d_logp, d_entropy, padding=-1):
    rows, vocab = x.shape
    logp = log_softmax(x, scale)
    p = np.exp(logp)
    plogp = np.where(p == 0, 0.0, p * np.where(p == 0, 0.0, logp))
    entropy = -plogp.sum(1, keepdims=True)
    grad = -d_entropy[:, None] * (plogp + p * entropy)
    for r in range(rows):
        for t, d in zip(tokens[r], d_logp[r]):
            if t != padding and 0 <= t < vocab:
                grad[r] -= d * p[r]
                grad[r, t] += d
    grad[np.isneginf(x).all(1)] = 0.0
    return grad * scale
