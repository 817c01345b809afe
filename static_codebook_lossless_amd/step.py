"""Binding of the norm, dropout and log-probability operators.

Argument marshalling only, with the conventions of ``q8``: plain tensors are
float32, float16 or bfloat16 rows of unit stride, wrong types, sizes, strides
or devices raise ``TypeError`` or ``ValueError``, and what the library itself
refuses raises ``PcError``.  Tensors of more than two dimensions count as rows
of their last one, and what is returned has their shape.

Tensors that a caller gives to be written (``out``, ``sum_out``,
``weight_out``) count as changed in place: where an autograd graph has saved
one, its backward pass raises torch's error instead of using what was written.
"""
from __future__ import annotations

import math
import operator

import torch

from ._lib import MaskArg, lib
from .q8 import Q8, _DTYPES, _FORMATS, PC_BF16, _code, _dtype, _launch, _rows, _same_device, _tokens

_Y = {None: None, "plain": 0, "stored": 1}


class DropoutMask:
    """Which elements a dropout drops: a share ``p`` of them, by their row and
    column and by ``seed`` and ``offset`` (64 bits each), with numbers that
    Philox4x32-10 gives for a counter.  It is stored nowhere; the backward pass
    takes the same object.  Two dropouts have different masks where their seed
    or offset differs: a layer's number and a step's make a good offset.

    ``seed`` may be an int64 device tensor of two numbers, the seed and one
    that is added to ``offset`` (both modulo 2**64): kernels read it where it
    is at the call, so a captured graph draws new masks when it changes.  The
    backward pass reads it too: its numbers have to stay until that has run
    (with several steps in flight, each takes a tensor of its own, or an
    ``offset``).  ``p`` is taken to the
    nearest multiple of 2**-16; what is not dropped is divided by the share
    that stays.  A mask is what it was made of: another ``p``, ``seed`` or
    ``offset`` is another object."""

    __slots__ = ("_p", "_seed", "_offset", "arg")

    def __init__(self, p, seed=0, offset=0):
        p = float(p)
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1], not %r" % p)
        offset = operator.index(offset)
        if not 0 <= offset < 1 << 64:
            raise ValueError("offset must have 64 bits")
        where = None
        if isinstance(seed, torch.Tensor):
            value, where = 0, _seed_address(seed)
        else:
            value = operator.index(seed)
            if not 0 <= value < 1 << 64:
                raise ValueError("seed must have 64 bits")
        self._p, self._seed, self._offset = p, seed, offset
        self.arg = MaskArg(p, value, offset, where)

    p = property(lambda self: self._p)
    seed = property(lambda self: self._seed)
    offset = property(lambda self: self._offset)


def _seed_address(seed):
    if not seed.is_cuda or seed.dtype != torch.int64 or seed.shape != (2,) or not seed.is_contiguous():
        raise TypeError("a seed on the device must be two contiguous int64")
    return seed.data_ptr()


def _mask(mask, device):
    """The mask's argument (None without one)."""
    if mask is None:
        return None
    if not isinstance(mask, DropoutMask):
        raise TypeError("mask must be a DropoutMask, not %s" % type(mask).__name__)
    if not mask.arg.d_random:
        return mask.arg
    # where the tensor is now: its memory may have been replaced since (``set_``, ``.data``)
    seed = mask._seed
    where = _seed_address(seed)
    if seed.device != device:
        raise ValueError("the mask's seed is on %s, not on %s" % (seed.device, device))
    return mask.arg if mask.arg.d_random == where else MaskArg(mask._p, 0, mask._offset, where)


def pc_dropout(x, mask: DropoutMask, out=None) -> torch.Tensor:
    """``x`` with ``mask``'s elements 0 and the others divided by the share
    that stays.  The backward pass is the same call on the gradient.  ``out``
    (of x's shape and dtype) receives it and may be ``x``."""
    kind = _dtype(x.dtype, "x")
    where, n, cols, ld = _flat(x, "x")
    if mask is None:
        raise TypeError("mask must be a DropoutMask")
    device = x.device
    arg = _mask(mask, device)
    given = out is not None
    out, to, ld_out = _like(out, x, x.dtype, cols, "out")
    _launch("pc_dropout", device, lib.pc_dropout, where, kind, n, cols, ld, arg, to, ld_out)
    if given:
        _written(out)
    return out


_DENSE = torch.contiguous_format


def _flat(t, what):
    """(address, rows, columns, row distance) of a plain device tensor seen as rows of its last dimension."""
    if t.is_contiguous() and t.is_cuda:
        shape = t.shape
        if len(shape) == 2:
            n, cols = shape
            return t.data_ptr(), n, cols, cols
        if shape:
            return t.data_ptr(), math.prod(shape[:-1]), shape[-1], shape[-1]
    rows, ld = _rows(t, what)
    return rows.data_ptr(), rows.shape[0], rows.shape[1], ld


def _like(out, x, dtype, cols, what):
    """(a tensor of x's shape, ``out`` itself where given, its address and row distance)"""
    if out is None:
        out = torch.empty_like(x, dtype=dtype, memory_format=_DENSE)
        return out, out.data_ptr(), cols
    where, ld = _same_rows(out, x, dtype, what)
    return out, where, ld


# kernels write by address: what torch's own in-place operations do to a tensor's version
_written = torch.autograd.graph.increment_version


def _same_rows(t, x, dtype, what):
    """(address, row distance) of a tensor of x's shape and of ``dtype``."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    shape = x.shape
    if t.shape != shape:
        raise ValueError("%s must be %s, not %s" % (what, list(shape), list(t.shape)))
    if t.device != x.device:
        raise ValueError("%s is on %s, not on %s" % (what, t.device, x.device))
    if t.is_contiguous() and shape:
        return t.data_ptr(), shape[-1]
    where, _, _, ld = _flat(t, what)
    return where, ld


def _weight(weight, cols, device, what="weight"):
    """(address, dtype) of a weight of cols numbers."""
    if weight is None:
        return None, 0
    kind = _dtype(weight.dtype, what)
    if weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError("%s must be %d contiguous numbers" % (what, cols))
    if weight.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, weight.device, device))
    return weight.data_ptr(), kind


def _a_row_each(x, n, device):
    """One float32 for each row of x."""
    if x.dim() == 2:  # of a size that is a number: a third quicker than of a shape
        return torch.empty(n, dtype=torch.float32, device=device)
    return torch.empty(x.shape[:-1], dtype=torch.float32, device=device)


class RmsNorm:
    """What ``pc_rmsnorm_store`` gives: ``q`` (the stored output, None without
    a format), ``y`` (None unless asked for), ``sum`` (x with dropout and
    residual; x itself without either) and ``rstd`` (one float32 a row)."""

    __slots__ = ("q", "y", "sum", "rstd")

    def __init__(self, q, y, sum, rstd):
        self.q, self.y, self.sum, self.rstd = q, y, sum, rstd


def pc_rmsnorm_store(x, weight=None, residual=None, mask=None, eps=1e-6, format="e4m3", counts=None, y=None,
                     dtype=None, sum_out=None) -> RmsNorm:
    """Root-mean-square norm of ``residual + mask(x)``, stored in 8 bits.

    ``sum = residual + mask(x)`` is rounded to the residual's dtype (x's own
    or float32; x's without one), and ``sum * rsqrt(mean(sum**2) + eps) * weight``
    is stored as ``pc_q8_store`` stores (``format``, ``counts``; None: not
    stored).  ``y`` asks for it in ``dtype`` (x's by default) too: "plain",
    rounded from 32 bits, or "stored", the values of the stored form, which are
    what a weight gradient will see.  ``sum_out`` receives the sum and may be
    the residual, or x where their dtypes agree."""
    kind = _dtype(x.dtype, "x")
    at, n, cols, ldx = _flat(x, "x")
    device = x.device
    eps = float(eps)
    arg = _mask(mask, device)
    w, w_kind = _weight(weight, cols, device)
    if y not in _Y:
        raise ValueError("y must be None, 'plain' or 'stored', not %r" % (y,))
    sum_dtype, res, ld_res = x.dtype, None, 0
    if residual is not None:
        if residual.dtype not in (x.dtype, torch.float32):
            raise TypeError("residual must be %s or float32, not %s" % (x.dtype, residual.dtype))
        sum_dtype = residual.dtype
        res, ld_res = _same_rows(residual, x, sum_dtype, "residual")
    total, where, ld_sum = x, None, 0
    if residual is not None or mask is not None:
        total, where, ld_sum = _like(sum_out, x, sum_dtype, cols, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual or a mask: the sum is x")
    q, sym, scale, code = None, None, None, 0
    if format is not None:
        code = _code(_FORMATS, format, "format")
        symbols = torch.empty(n, cols, dtype=torch.uint8, device=device)
        scales = torch.empty(n, -(-cols // 32), dtype=torch.uint8, device=device)
        q = Q8._dense(symbols, scales, format, n, cols, code)
        sym, scale = q.arg.sym, q.arg.scale
    elif y == "stored" or counts is not None:
        raise ValueError("stored values and counts need a format")
    if counts is not None:
        if counts.dtype != torch.int64 or counts.shape != (256,) or not counts.is_contiguous():
            raise TypeError("counts must be 256 contiguous int64")
        _same_device(x, counts, "counts")
    out, to, to_kind = None, None, kind
    if y is not None:
        if dtype is not None:
            to_kind = _dtype(dtype, "dtype")
        out = torch.empty_like(x, dtype=dtype, memory_format=_DENSE)
        to = out.data_ptr()
    rstd = _a_row_each(x, n, device)
    _launch("pc_rmsnorm_store", device, lib.pc_rmsnorm_store, at, kind, n, cols, ldx, res,
            _DTYPES[sum_dtype], ld_res, arg, w, w_kind, eps, where, ld_sum, code, sym, scale,
            None if counts is None else counts.data_ptr(), to, to_kind, cols, int(y == "stored"), rstd.data_ptr())
    if sum_out is not None:
        _written(sum_out)
    return RmsNorm(q, out, total, rstd)


class RmsNormGrads:
    """Gradients of ``pc_rmsnorm_store``'s inputs: ``residual`` (of the sum as
    well), ``x`` (the same tensor where there is no mask and one dtype) and
    ``weight`` (None without a weight)."""

    __slots__ = ("residual", "x", "weight")

    def __init__(self, residual, x, weight):
        self.residual, self.x, self.weight = residual, x, weight


def pc_rmsnorm_backward_workspace_bytes(rows, cols):
    return int(lib.pc_rmsnorm_backward_workspace_bytes(rows, cols))


def pc_rmsnorm_backward(dy, sum, weight, rstd, d_sum=None, mask=None, dtype=None, weight_dtype=torch.float32,
                        weight_out=None, accumulate=False) -> RmsNormGrads:
    """Backward pass of ``pc_rmsnorm_store`` for the gradient ``dy`` of its y.

    ``sum`` is the forward pass's, or a ``Q8`` of it; ``d_sum`` the gradient
    that reaches it on the residual's way, in its dtype; ``mask`` the forward
    pass's.  ``dtype`` is the residual's dtype where sum is a ``Q8`` (d_sum's
    or dy's by default).  ``weight_out`` (of weight_dtype) receives the
    weight's gradient; with ``accumulate`` it is added there."""
    kind, out_kind = _dtype(dy.dtype, "dy"), _dtype(weight_dtype, "weight_dtype")
    at, n, cols, ld_dy = _flat(dy, "dy")
    device = dy.device
    arg = _mask(mask, device)
    w, w_kind = _weight(weight, cols, device)
    kept, kept_ld, stored = None, 0, None
    if isinstance(sum, Q8):
        if sum.symbols.shape != (n, cols):
            raise ValueError("sum must be [%d, %d], not %s" % (n, cols, list(sum.symbols.shape)))
        _same_device(dy, sum.symbols, "sum")
        stored = sum.arg
        if dtype is None:
            dtype = dy.dtype if d_sum is None else d_sum.dtype
    else:
        if dtype is None:
            dtype = sum.dtype
        kept, kept_ld = _same_rows(sum, dy, dtype, "sum")
    if dtype not in (dy.dtype, torch.float32):
        raise TypeError("the residual's dtype must be %s or float32, not %s" % (dy.dtype, dtype))
    if rstd.dtype != torch.float32 or rstd.numel() != n or not rstd.is_contiguous():
        raise TypeError("rstd must be %d contiguous float32" % n)
    _same_device(dy, rstd, "rstd")
    ds, ld_ds = (None, 0) if d_sum is None else _same_rows(d_sum, dy, dtype, "d_sum")
    if weight is None and weight_out is not None:
        raise ValueError("weight_out needs a weight")
    if accumulate and weight_out is None:
        raise ValueError("accumulate needs weight_out")
    if weight_out is not None:
        if weight_out.dtype != weight_dtype:
            raise TypeError("weight_out must be %s, not %s" % (weight_dtype, weight_out.dtype))
        _weight(weight_out, cols, device, "weight_out")
    residual = torch.empty_like(dy, dtype=dtype, memory_format=_DENSE)
    x, d_x = residual, None
    if mask is not None or dtype != dy.dtype:
        x = torch.empty_like(dy, memory_format=_DENSE)
        d_x = x.data_ptr()
    d_weight, ws, need = weight_out, None, 0
    if weight is not None:
        if d_weight is None:
            d_weight = torch.empty(cols, dtype=weight_dtype, device=device)
        need = lib.pc_rmsnorm_backward_workspace_bytes(n, cols)
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch("pc_rmsnorm_backward", device, lib.pc_rmsnorm_backward, at, kind, n, cols, ld_dy, kept,
            _DTYPES[dtype], kept_ld, stored, w, w_kind, rstd.data_ptr(), ds, ld_ds, arg, residual.data_ptr(), cols,
            d_x, cols, None if d_weight is None else d_weight.data_ptr(), out_kind, int(accumulate),
            None if ws is None else ws.data_ptr(), need)
    if weight_out is not None:
        _written(weight_out)
    return RmsNormGrads(residual, x, d_weight)


class LogProbs:
    """What ``pc_logprobs`` gives: ``logp`` (of the tokens' shape, None without
    tokens), ``top_index`` and ``top_logp`` ([..., top], None without), and
    ``stats`` ([rows, 4] float32, which the backward pass takes), out of which
    ``entropy`` and ``lse`` (the logarithm of the sum of exponentials) are views."""

    __slots__ = ("logp", "top_index", "top_logp", "stats", "_lead")

    def __init__(self, logp, top_index, top_logp, stats, lead):
        self.logp, self.top_index, self.top_logp, self.stats, self._lead = logp, top_index, top_logp, stats, lead

    def _column(self, k):
        strides, s = [], 4
        for size in reversed(self._lead):
            strides.append(s)
            s *= size
        return self.stats.as_strided(self._lead, strides[::-1], self.stats.storage_offset() + k)

    @property
    def entropy(self):
        return self._column(2)

    @property
    def lse(self):
        return self._column(3)


def pc_logprobs_workspace_bytes(rows, vocab, top=0, dtype=PC_BF16):
    return int(lib.pc_logprobs_workspace_bytes(rows, vocab, top, dtype))


def _padding(padding):
    padding = operator.index(padding)
    if not -1 << 63 <= padding < 1 << 63:
        raise ValueError("padding must have 64 bits, with its sign")
    return padding


def _picked(tokens, lead, device):
    """(tokens, how many each row has) for rows of the shape ``lead``."""
    tokens = _tokens(tokens, device)
    if tokens.shape == lead:
        return tokens, 1
    if tokens.shape[:-1] != lead:
        raise ValueError("tokens must be %s or that with one more dimension, not %s" % (list(lead), list(tokens.shape)))
    return tokens, tokens.shape[-1]


def pc_logprobs(logits, tokens=None, top=0, scale=1.0, padding=-1, status=None) -> LogProbs:
    """Log probabilities of ``tokens`` under ``softmax(scale * logits)``, its
    entropy, and the ``top`` most probable tokens.

    ``logits`` is [..., vocab], ``tokens`` [...] or, with several for each row
    (at most 64), [..., m].  A token equal to ``padding`` or outside the
    vocabulary gets 0 and, unless it is the padding, sets ``status`` (int32 [1]
    on the device, zeroed by the caller) to ``PC_ERR_INVALID_ARG``.  Equal
    logits are ordered by their index."""
    kind, scale, padding, top = _dtype(logits.dtype, "logits"), float(scale), _padding(padding), operator.index(top)
    at, n, vocab, ld = _flat(logits, "logits")
    device, lead = logits.device, logits.shape[:-1]
    logp, where, m, width = None, None, 0, 8
    if tokens is not None:
        tokens, m = _picked(tokens, lead, device)
        width = tokens.element_size()
        logp = torch.empty_like(tokens, dtype=torch.float32)
        where = tokens.data_ptr()
    if top < 0:
        raise ValueError("top is negative")
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != device):
        raise TypeError("status must be one int32 on the logits' device")
    index = value = None
    if top:
        index = torch.empty(*lead, top, dtype=torch.int64, device=device)
        value = torch.empty_like(index, dtype=torch.float32)
    stats = torch.empty(n, 4, dtype=torch.float32, device=device)
    need = lib.pc_logprobs_workspace_bytes(n, vocab, top, kind)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch("pc_logprobs", device, lib.pc_logprobs, at, kind, n, vocab, ld, scale, where, width, m, padding,
            None if logp is None else logp.data_ptr(), top, None if index is None else index.data_ptr(),
            None if value is None else value.data_ptr(), stats.data_ptr(), None if status is None else status.data_ptr(),
            None if ws is None else ws.data_ptr(), need)
    return LogProbs(logp, index, value, stats, lead)


def pc_logprobs_backward(logits, stats, tokens=None, d_logp=None, d_entropy=None, scale=1.0, padding=-1,
                         out=None) -> torch.Tensor:
    """Gradient of the logits from those of ``pc_logprobs``'s log probabilities
    (``d_logp``, of the tokens' shape) and entropy (``d_entropy``), both
    float32.  ``stats``, ``tokens``, ``scale`` and ``padding`` are the forward
    pass's.  ``out`` (of the logits' shape and dtype) receives it and may be
    ``logits``, where nothing reads these any more: no second backward pass, no
    other loss that has saved them."""
    kind, scale, padding = _dtype(logits.dtype, "logits"), float(scale), _padding(padding)
    at, n, vocab, ld = _flat(logits, "logits")
    device, lead = logits.device, logits.shape[:-1]
    if stats.dtype != torch.float32 or stats.shape != (n, 4) or not stats.is_contiguous():
        raise TypeError("stats must be [%d, 4] contiguous float32" % n)
    _same_device(logits, stats, "stats")
    where, m, width = None, 0, 8
    if (tokens is None) != (d_logp is None):
        raise ValueError("tokens and d_logp go together")
    if tokens is not None:
        tokens, m = _picked(tokens, lead, device)
        width = tokens.element_size()
        where = tokens.data_ptr()
        d_logp = _gradient(d_logp, tokens.shape, logits, "d_logp")
    if d_entropy is not None:
        d_entropy = _gradient(d_entropy, lead, logits, "d_entropy")
    given = out is not None
    out, to, ld_out = _like(out, logits, logits.dtype, vocab, "out")
    _launch("pc_logprobs_backward", device, lib.pc_logprobs_backward, at, kind, n, vocab, ld, scale,
            stats.data_ptr(), where, width, m, padding, None if d_logp is None else d_logp.data_ptr(),
            None if d_entropy is None else d_entropy.data_ptr(), to, ld_out)
    if given:
        _written(out)
    return out


def _gradient(d, shape, logits, what):
    if d.dtype != torch.float32:
        raise TypeError("%s must be float32, not %s" % (what, d.dtype))
    if d.shape != shape:
        raise ValueError("%s must be %s, not %s" % (what, list(shape), list(d.shape)))
    _same_device(logits, d, what)
    return d.contiguous()
