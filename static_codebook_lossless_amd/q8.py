"""Binding of the stored-tensor and embedding operators.

Argument marshalling only, as in ``_lib``: torch tensors supply device memory,
the current torch stream of the tensors' device supplies the HIP stream.
Plain tensors are float32, float16 or bfloat16 with a unit stride along the
last dimension; their leading dimensions have to collapse into rows of one
distance (``view(-1, cols)``).  Wrong types, sizes, strides or devices raise
``TypeError`` or ``ValueError``; what the library itself refuses raises
``PcError``.
"""
from __future__ import annotations

import math
import operator

import torch

from ._lib import StoredArg, _check, lib

PC_F32, PC_F16, PC_BF16 = range(3)
PC_Q8_E4M3, PC_Q8_INT8 = range(2)
PC_ACT_SILU, PC_ACT_GELU, PC_ACT_GELU_TANH = range(3)
PC_Q8_GROUP = 32

_DTYPES = {torch.float32: PC_F32, torch.float16: PC_F16, torch.bfloat16: PC_BF16}
_FORMATS = {"e4m3": PC_Q8_E4M3, "int8": PC_Q8_INT8}
_ACTS = {"silu": PC_ACT_SILU, "gelu": PC_ACT_GELU, "gelu_tanh": PC_ACT_GELU_TANH}


def _dtype(dtype, what):
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise TypeError("%s must be float32, float16 or bfloat16, not %s" % (what, dtype)) from None


def _code(names, name, what):
    try:
        return names[name]
    except KeyError:
        raise ValueError("%s must be one of %s, not %r" % (what, ", ".join(names), name)) from None


def _rows(t, what):
    """(t as rows, its row distance) of a plain device tensor of at least one dimension."""
    if not t.is_cuda:
        raise TypeError("%s must be a device tensor" % what)
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError("%s must have a dimension" % what)
        try:
            t = t.view(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError:
            raise ValueError("the leading dimensions of %s do not collapse into rows" % what) from None
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit stride along its last dimension" % what)
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError("the rows of %s overlap" % what)
    return t, ld


def _same_device(a, b, what):
    if a.device != b.device:
        raise ValueError("%s is on %s, not on %s" % (what, b.device, a.device))


# the current stream's handle without the Stream object that
# torch.cuda.current_stream builds around it (2 us of a 9 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(what, device, fn, *args):
    """Call ``fn`` on the device's current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(st, what)


class Q8:
    """A tensor stored in 8 bits.

    ``symbols``  uint8 [rows, cols]: e4m3 or int8 elements (``format``)
    ``scales``   uint8 [rows, ceil(cols / 32)]: codes; an element stands for
                 ``element * 2**(code - 127)``

    Both need unit stride along the rows.  Dense symbols are the bytes that
    ``pc_encode`` takes: ``pc_encode(cb, q.symbols, chunk)``; and what
    ``pc_decode`` gives back becomes a stored tensor again with
    ``q.with_symbols(bytes)``.
    """

    __slots__ = ("symbols", "scales", "format", "arg")

    def __init__(self, symbols, scales, format="e4m3"):
        code = _code(_FORMATS, format, "format")
        if symbols.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("symbols and scales must be uint8")
        if symbols.dim() != 2 or scales.dim() != 2:
            raise ValueError("symbols and scales must have two dimensions")
        rows, cols = symbols.shape
        groups = -(-cols // PC_Q8_GROUP)
        if scales.shape != (rows, groups):
            raise ValueError("scales must be [rows, ceil(cols / 32)] = [%d, %d], not %s"
                             % (rows, groups, list(scales.shape)))
        if symbols.is_cuda and symbols.is_contiguous() and scales.is_contiguous():
            ld, ld_scale = cols, groups
        else:
            symbols, ld = _rows(symbols, "symbols")
            scales, ld_scale = _rows(scales, "scales")
        _same_device(symbols, scales, "scales")
        self.symbols, self.scales, self.format = symbols, scales, format
        self.arg = StoredArg(symbols.data_ptr(), scales.data_ptr(), rows, cols, ld, ld_scale, code, 0)

    @classmethod
    def _dense(cls, symbols, scales, format, rows, cols, code):
        """A stored tensor of two dense tensors just allocated for it."""
        q = cls.__new__(cls)
        q.symbols, q.scales, q.format = symbols, scales, format
        q.arg = StoredArg(symbols.data_ptr(), scales.data_ptr(), rows, cols, cols, -(-cols // PC_Q8_GROUP), code, 0)
        return q

    @property
    def shape(self):
        return self.symbols.shape

    @property
    def device(self):
        return self.symbols.device

    def with_symbols(self, symbols):
        """The same tensor with its symbols in other memory (decoded bytes)."""
        try:
            symbols = symbols.view(self.symbols.shape)
        except RuntimeError:
            raise ValueError("symbols of %s cannot be seen as %s"
                             % (list(symbols.shape), list(self.symbols.shape))) from None
        return Q8(symbols, self.scales, self.format)

    def columns(self, begin, end):
        """A view of columns [begin, end); begin is a multiple of 32."""
        cols = self.symbols.shape[1]
        if begin % PC_Q8_GROUP or not 0 <= begin <= end <= cols or (end % PC_Q8_GROUP and end != cols):
            raise ValueError("columns begin and end at multiples of 32 (or at the tensor's end)")
        return Q8(self.symbols[:, begin:end], self.scales[:, begin // PC_Q8_GROUP:-(-end // PC_Q8_GROUP)],
                  self.format)


def _stored(q, what):
    if not isinstance(q, Q8):
        raise TypeError("%s must be a Q8, not %s" % (what, type(q).__name__))


def pc_q8_store(x, format="e4m3", counts=None) -> Q8:
    """Store ``x`` in 8 bits with one scale for every 32 columns.  ``counts``
    (int64 [256] on the device) gets the histogram of the symbols added, in
    the same pass.  x of more than two dimensions is stored as rows of its
    last one.  Infinities and NaN read back as NaN; finite magnitudes that
    round to 2**128 (the largest finite float32 and bfloat16 do) read back as
    infinity."""
    code, kind = _code(_FORMATS, format, "format"), _dtype(x.dtype, "x")
    x, ld = _rows(x, "x")
    rows, cols = x.shape
    if counts is not None:
        if counts.dtype != torch.int64 or counts.shape != (256,) or not counts.is_contiguous():
            raise TypeError("counts must be 256 contiguous int64")
        _same_device(x, counts, "counts")
    device = x.device
    symbols = torch.empty((rows, cols), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, -(-cols // PC_Q8_GROUP)), dtype=torch.uint8, device=device)
    q = Q8._dense(symbols, scales, format, rows, cols, code)
    _launch("pc_q8_store", device, lib.pc_q8_store, x.data_ptr(), kind, rows, cols, ld, code, q.arg.sym, q.arg.scale,
            None if counts is None else counts.data_ptr())
    return q


def _output(out, shape, dtype, device, what="out"):
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        return out, shape[1]
    if out.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, out.dtype))
    rows, ld = _rows(out, what)
    if tuple(rows.shape) != tuple(shape):
        raise ValueError("%s must be %s, not %s" % (what, list(shape), list(out.shape)))
    if out.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, out.device, device))
    return out, ld


def pc_q8_load(q: Q8, dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """The values of a stored tensor, rounded to ``dtype`` (``out``: where to, of that dtype)."""
    _stored(q, "q")
    kind = _dtype(dtype, "dtype")
    out, ld = _output(out, tuple(q.symbols.shape), dtype, q.device)
    _launch("pc_q8_load", q.device, lib.pc_q8_load, q.arg, out.data_ptr(), kind, ld)
    return out


class GluGrads:
    """Gradients of a gated activation: ``gate``, ``up`` (None without a
    gate), the recomputed ``h`` (None unless asked for), and, where gate and
    up were one tensor, ``packed``: both gradients side by side."""

    __slots__ = ("_gate", "_up", "h", "packed")

    def __init__(self, gate, up, h, packed=None):
        self._gate, self._up, self.h, self.packed = gate, up, h, packed

    @property
    def gate(self):
        return self._gate if self.packed is None else self.packed[:, :self.packed.shape[1] // 2]

    @property
    def up(self):
        return self._up if self.packed is None else self.packed[:, self.packed.shape[1] // 2:]


def pc_q8_glu_backward(dh, gate: Q8, up: Q8 | None = None, act="silu", with_h=False) -> GluGrads:
    """Backward pass of ``h = act(gate) * up`` from stored gate and up.

    ``dh`` is [rows, cols].  Without ``up``, a ``gate`` of 2 * cols columns
    holds gate and up side by side (cols a multiple of 32), and one of cols
    columns is an activation without a gate, ``h = act(gate)``.  Gradients and
    ``h`` are [rows, cols] of dh's dtype (a dh of more dimensions counts as
    rows of its last one)."""
    _stored(gate, "gate")
    if up is not None:
        _stored(up, "up")
    kind, a = _dtype(dh.dtype, "dh"), _code(_ACTS, act, "act")
    x, ld = _rows(dh, "dh")
    rows, cols = x.shape
    _same_device(x, gate.symbols, "gate")
    packed = None
    if up is not None:
        if up.symbols.shape != (rows, cols) or gate.symbols.shape != (rows, cols):
            raise ValueError("gate and up must be [%d, %d] as dh is" % (rows, cols))
        if up.format != gate.format:
            raise ValueError("gate and up must have one format")
        _same_device(x, up.symbols, "up")
        g, u = gate.arg, up.arg
    elif cols and gate.symbols.shape == (rows, 2 * cols):
        if cols % PC_Q8_GROUP:
            raise ValueError("gate and up in one tensor need a multiple of 32 columns each, not %d" % cols)
        g, u = StoredArg.from_buffer_copy(gate.arg), StoredArg.from_buffer_copy(gate.arg)
        g.cols = u.cols = cols
        u.sym = (gate.arg.sym or 0) + cols
        u.scale = (gate.arg.scale or 0) + cols // PC_Q8_GROUP
        packed = torch.empty((rows, 2 * cols), dtype=x.dtype, device=x.device)
    elif gate.symbols.shape == (rows, cols):
        g, u = gate.arg, None
    else:
        raise ValueError("gate must be [%d, %d], or twice as wide with up beside it" % (rows, cols))
    h = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if with_h else None
    if packed is not None:
        dg = du = None
        pg, ld_out = packed.data_ptr(), 2 * cols
        pu = pg + cols * packed.element_size()
    else:
        dg = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        du = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if up is not None else None
        pg, ld_out = dg.data_ptr(), cols
        pu = None if du is None else du.data_ptr()
    _launch("pc_q8_glu_backward", x.device, lib.pc_q8_glu_backward, x.data_ptr(), kind, ld, g, u, a, pg, ld_out, pu,
            ld_out, None if h is None else h.data_ptr(), cols)
    return GluGrads(dg, du, h, packed)


def pc_q8_weight_grad_workspace_bytes(rows, n_out, n_in, dy_dtype=PC_BF16):
    return int(lib.pc_q8_weight_grad_workspace_bytes(rows, n_out, n_in, dy_dtype))


def pc_q8_weight_grad(dy, x: Q8, dtype=torch.float32, out=None, accumulate=False) -> torch.Tensor:
    """``dy^T @ x`` for a stored ``x``: [n_out, n_in] of ``dtype``.  ``out``
    (of that dtype) receives it; with ``accumulate`` it is added there."""
    _stored(x, "x")
    kind, out_kind = _dtype(dy.dtype, "dy"), _dtype(dtype, "dtype")
    dy, ld = _rows(dy, "dy")
    _same_device(dy, x.symbols, "x")
    rows, n_out = dy.shape
    n_in = x.symbols.shape[1]
    if x.symbols.shape[0] != rows:
        raise ValueError("dy has %d rows, x has %d" % (rows, x.symbols.shape[0]))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out, ld_out = _output(out, (n_out, n_in), dtype, dy.device)
    need = lib.pc_q8_weight_grad_workspace_bytes(rows, n_out, n_in, kind)
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    _launch("pc_q8_weight_grad", dy.device, lib.pc_q8_weight_grad, dy.data_ptr(), kind, ld, n_out, x.arg,
            out.data_ptr(), out_kind, ld_out, int(accumulate), None if ws is None else ws.data_ptr(), need)
    return out


def _tokens(tokens, device):
    if tokens.dtype not in (torch.int64, torch.int32):
        raise TypeError("tokens must be int64 or int32, not %s" % tokens.dtype)
    if tokens.device != device:
        raise ValueError("tokens is on %s, not on %s" % (tokens.device, device))
    return tokens.contiguous()


def pc_embed(tokens, table, scale=1.0, dtype=None, out=None, status=None) -> torch.Tensor:
    """``scale * table[tokens]``: [*tokens.shape, dim] of ``dtype`` (the
    table's own by default, bfloat16 for a stored table).  ``table`` is
    [vocab, dim], plain or a ``Q8``.  A token outside the table gives a row
    of zeros and, where ``status`` (int32 [1] on the device, zeroed by the
    caller) is given, sets it to ``PC_ERR_INVALID_ARG``."""
    stored, scale = isinstance(table, Q8), float(scale)
    rows, ld = (table.symbols, 0) if stored else _rows(table, "table")
    if not stored and table.dim() != 2:
        raise ValueError("table must have two dimensions")
    if dtype is None:
        dtype = torch.bfloat16 if stored else table.dtype
    kind = _dtype(dtype, "dtype")
    vocab, dim = rows.shape
    tokens = _tokens(tokens, rows.device)
    n = tokens.numel()
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != rows.device):
        raise TypeError("status must be one int32 on the table's device")
    if out is None:
        out, ld_out = torch.empty((*tokens.shape, dim), dtype=dtype, device=rows.device), dim
    else:
        if tuple(out.shape) != (*tokens.shape, dim):
            raise ValueError("out must be %s, not %s" % ([*tokens.shape, dim], list(out.shape)))
        if out.dim() == 1:
            out, ld_out = _output(out.view(1, dim), (1, dim), dtype, rows.device)[0].view(dim), dim
        else:
            out, ld_out = _output(out, (n, dim), dtype, rows.device)
    where = None if status is None else status.data_ptr()
    if stored:
        _launch("pc_embed_q8", rows.device, lib.pc_embed_q8, tokens.data_ptr(), tokens.element_size(), n, table.arg,
                scale, out.data_ptr(), kind, ld_out, where)
    else:
        _launch("pc_embed", rows.device, lib.pc_embed, tokens.data_ptr(), tokens.element_size(), n, rows.data_ptr(),
                _dtype(table.dtype, "table"), vocab, dim, ld, scale, out.data_ptr(), kind, ld_out, where)
    return out


def pc_embed_q8(tokens, table: Q8, scale=1.0, dtype=torch.bfloat16, out=None, status=None) -> torch.Tensor:
    """``pc_embed`` of a stored table."""
    _stored(table, "table")
    return pc_embed(tokens, table, scale, dtype, out, status)


def pc_embed_backward_workspace_bytes(n, dim, vocab):
    return int(lib.pc_embed_backward_workspace_bytes(n, dim, vocab))


def pc_embed_backward(dy, tokens, vocab, scale=1.0, dtype=torch.float32, padding=-1, out=None,
                      accumulate=False) -> torch.Tensor:
    """Gradient of the table: [vocab, dim] of ``dtype``, row v the sum of
    ``scale * dy`` over the tokens equal to v, summed in their order.  Tokens
    outside the table or equal to ``padding`` add nothing.  ``out`` (of that
    dtype) receives it; with ``accumulate`` it is added there."""
    kind, out_kind = _dtype(dy.dtype, "dy"), _dtype(dtype, "dtype")
    scale, padding = float(scale), operator.index(padding)
    if dy.shape[:-1] != tokens.shape:
        raise ValueError("dy must be [*tokens.shape, dim]")
    dy, ld = _rows(dy, "dy")
    n, dim = dy.shape
    tokens = _tokens(tokens, dy.device)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if vocab < 0:
        raise ValueError("vocab is negative")
    out, ld_out = _output(out, (vocab, dim), dtype, dy.device)
    need = lib.pc_embed_backward_workspace_bytes(n, dim, vocab)
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    _launch("pc_embed_backward", dy.device, lib.pc_embed_backward, dy.data_ptr(), kind, ld, tokens.data_ptr(),
            tokens.element_size(), n, dim, vocab, padding, scale, out.data_ptr(), out_kind, ld_out, int(accumulate),
            None if ws is None else ws.data_ptr(), need)
    return out
