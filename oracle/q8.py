"""Plain 64-bit forms of the stored-tensor and embedding operators (numpy).

Written from the definitions in include/pc.h, element by element where that
is the plainest; shares no code or tables with the library.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
MOST = {"e4m3": 448.0, "int8": 127.0}
NAN_BYTE = {"e4m3": 0x7F, "int8": 0x80}
MIN_EXPONENT = -117


def element(byte: int, fmt: str) -> float:
    """The number a symbol stands for before scaling (OCP E4M3FN: 4 exponent
    bits of bias 7, 3 mantissa bits, S.1111.111 is NaN; int8: two's
    complement, -128 is NaN)."""
    if fmt == "int8":
        return math.nan if byte == 0x80 else float(byte - 256 if byte > 127 else byte)
    sign, e, m = -1.0 if byte & 0x80 else 1.0, byte >> 3 & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * math.ldexp(m, -9) if e == 0 else sign * math.ldexp(8 + m, e - 10)


def elements(fmt: str) -> np.ndarray:
    return np.array([element(b, fmt) for b in range(256)])


def nearest_byte(y: float, fmt: str) -> int:
    """The symbol nearest to y, ties to the even significand (for int8 the
    even number), zeros keeping their sign in e4m3."""
    if fmt == "int8":
        lo = math.floor(y)
        d = y - lo
        v = lo if d < 0.5 or (d == 0.5 and lo % 2 == 0) else lo + 1
        return v & 0xFF
    sign = 0x80 if math.copysign(1.0, y) < 0 else 0
    y = abs(y)
    best = None
    for b in range(0x7F):  # 0 .. 448 in ascending order
        d = abs(element(b, fmt) - y)
        if best is None or d < best[0] or (d == best[0] and b % 2 == 0):
            best = (d, b)
    return sign | best[1]


def exponent_for(top: float, fmt: str) -> int:
    k = MIN_EXPONENT
    while top > MOST[fmt] * 2.0 ** k:
        k += 1
    return k


def exponent_near(top: float, fmt: str) -> int:
    """``exponent_for``, starting its search near the answer."""
    if top == 0.0:
        return MIN_EXPONENT
    k = max(MIN_EXPONENT, math.frexp(top)[1] - 12)
    while top > MOST[fmt] * 2.0 ** k:
        k += 1
    return k


def nearest_bytes(y: np.ndarray, fmt: str) -> np.ndarray:
    """``nearest_byte`` of an array: by the number of midpoints between
    neighbouring magnitudes that lie below, those met exactly going to the even one."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.rint(y).astype(np.int64).astype(np.uint8)
    e = elements(fmt)[:0x7F]
    middle = (e[1:] + e[:-1]) / 2
    low, high = np.searchsorted(middle, np.abs(y), "left"), np.searchsorted(middle, np.abs(y), "right")
    b = np.where((low != high) & (low % 2 == 1), high, low)
    return (b | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def store(x: np.ndarray, fmt: str):
    """(symbols uint8 [rows, cols], codes uint8 [rows, groups]) of x."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    finite = np.isfinite(x)
    top = np.zeros((rows, groups * GROUP))
    top[:, :cols] = np.where(finite, np.abs(x), 0.0)
    top = top.reshape(rows, groups, GROUP).max(axis=2) if cols else np.zeros((rows, 0))
    # a number m 2^e with 1/2 <= m < 1 needs the exponent of M, or one more
    k = np.array([[exponent_near(v, fmt) for v in r] for r in top], dtype=np.int64).reshape(rows, groups)
    wide = np.repeat(k, GROUP, axis=1)[:, :cols]
    sym = nearest_bytes(np.where(finite, x, 0.0) * np.exp2(-wide), fmt)
    return np.where(finite, sym, NAN_BYTE[fmt]).astype(np.uint8), (k + 127).astype(np.uint8)


def load(sym: np.ndarray, codes: np.ndarray, fmt: str) -> np.ndarray:
    scale = np.exp2(codes.astype(np.float64) - 127.0)
    return elements(fmt)[sym] * np.repeat(scale, GROUP, axis=1)[:, :sym.shape[1]]


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        return g / (1.0 + np.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + _erf(g / math.sqrt(2.0)))
    return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def act_slope(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(g / math.sqrt(2.0))) + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = np.tanh(a * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * g * g)


def glu_backward(dh, g, u, name):
    """(d_gate, d_up, h) of h = act(g) u."""
    return dh * u * act_slope(name, g), dh * act(name, g), act(name, g) * u


def weight_grad(dy, x):
    return np.asarray(dy, dtype=np.float64).T @ np.asarray(x, dtype=np.float64)


def embed(tokens, table, scale):
    t = np.asarray(tokens).reshape(-1)
    out = np.zeros((t.size, table.shape[1]))
    for i, v in enumerate(t):
        if 0 <= v < table.shape[0]:
            out[i] = table[v] * scale
    return out.reshape(*np.shape(tokens), table.shape[1])


def embed_backward(dy, tokens, vocab, scale, padding=-1):
    """(gradient, sum of magnitudes, number of terms) of each row."""
    t = np.asarray(tokens).reshape(-1)
    dy = np.asarray(dy, dtype=np.float64).reshape(t.size, -1)
    grad = np.zeros((vocab, dy.shape[1]))
    size, terms = np.zeros_like(grad), np.zeros(vocab, dtype=np.int64)
    for i, v in enumerate(t):
        if 0 <= v < vocab and v != padding:
            grad[v] += dy[i] * scale
            size[v] += np.abs(dy[i] * scale)
            terms[v] += 1
    return grad, size, terms
