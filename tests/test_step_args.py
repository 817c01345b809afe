"""Refusals of the norm, dropout and log-probability operators, on the CPU:
every call is rejected, or has nothing to do, before the library touches the
device (fake addresses, never dereferenced)."""
import ctypes as C
import math

import pytest
import torch

import static_codebook_lossless_amd as pc
from static_codebook_lossless_amd._lib import MaskArg, StoredArg

lib = pc._lib.lib
A = 1 << 20
BAD, BIG, SMALL, OK = pc.PC_ERR_INVALID_ARG, pc.PC_ERR_UNSUPPORTED, pc.PC_ERR_CAPACITY, pc.PC_OK
F32, F16, BF16 = pc.PC_F32, pc.PC_F16, pc.PC_BF16


def mask(p=0.5, where=None):
    return MaskArg(p, 1, 2, where)


def q8(rows=4, cols=64, sym=A, scale=A, ld=None, lds=None, fmt=0):
    return StoredArg(sym, scale, rows, cols, cols if ld is None else ld, -(-cols // 32) if lds is None else lds, fmt, 0)


def dropout(x=A, dtype=BF16, rows=4, cols=64, ld=64, m=mask(), out=2 * A, ldo=64):
    return lib.pc_dropout(x, dtype, rows, cols, ld, m, out, ldo, None)


def norm(x=A, dtype=BF16, rows=4, cols=64, ld=64, res=2 * A, sum_dtype=BF16, ldr=64, m=None, w=3 * A, wd=F32, eps=1e-6,
         total=4 * A, lds=64, fmt=0, sym=5 * A, scale=6 * A, counts=None, y=7 * A, yd=BF16, ldy=64, stored=0,
         rstd=8 * A):
    return lib.pc_rmsnorm_store(x, dtype, rows, cols, ld, res, sum_dtype, ldr, m, w, wd, eps, total, lds, fmt, sym, scale,
                                counts, y, yd, ldy, stored, rstd, None)


def back(dy=A, dtype=BF16, rows=4, cols=64, ld=64, total=2 * A, sum_dtype=BF16, lds=64, q=None, w=3 * A, wd=F32,
         rstd=4 * A, ds=5 * A, ldds=64, m=None, dres=6 * A, ldr=64, dx=7 * A, ldx=64, dw=8 * A, dwd=F32, acc=0, ws=9 * A,
         wsb=1 << 40):
    return lib.pc_rmsnorm_backward(dy, dtype, rows, cols, ld, total, sum_dtype, lds, q, w, wd, rstd, ds, ldds, m, dres, ldr,
                                   dx, ldx, dw, dwd, acc, ws, wsb, None)


def logp(x=A, dtype=BF16, rows=4, vocab=100, ld=100, scale=1.0, tok=2 * A, tb=8, m=1, out=3 * A, top=5, index=4 * A,
         value=5 * A, stats=6 * A, status=None, ws=7 * A, wsb=1 << 40):
    return lib.pc_logprobs(x, dtype, rows, vocab, ld, scale, tok, tb, m, -1, out, top, index, value, stats, status, ws, wsb,
                           None)


def logp_back(x=A, dtype=BF16, rows=4, vocab=100, ld=100, scale=1.0, stats=2 * A, tok=3 * A, tb=8, m=1, d=4 * A, de=5 * A,
              out=6 * A, ldo=100):
    return lib.pc_logprobs_backward(x, dtype, rows, vocab, ld, scale, stats, tok, tb, m, -1, d, de, out, ldo, None)


BAD_MASKS = [mask(-0.1), mask(1.1), mask(math.nan), mask(math.inf), mask(0.5, A + 4)]


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=A + 1), dict(dtype=3), dict(ld=63), dict(out=None), dict(out=A + 1),
                                dict(ldo=63), dict(m=None), dict(out=A, ldo=128)] + [dict(m=m) for m in BAD_MASKS])
def test_dropout_refuses(kw):
    assert dropout(**kw) == BAD


def test_dropout_sizes():
    assert dropout(rows=0, x=None, out=None) == OK and dropout(cols=0, x=None, out=None) == OK
    assert dropout(cols=1 << 31, ld=1 << 31, ldo=1 << 31) == BIG
    assert dropout(rows=1 << 40) == BIG and dropout(rows=1 << 20, ld=1 << 45) == BIG
    assert dropout(rows=1 << 20, ldo=1 << 45) == BIG


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=A + 1), dict(dtype=3), dict(sum_dtype=F16), dict(sum_dtype=7),
                                dict(dtype=F32), dict(ld=63), dict(res=2 * A + 1), dict(ldr=63), dict(wd=4), dict(w=3 * A + 2),
                                dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(lds=63),
                                dict(total=4 * A + 1), dict(fmt=2), dict(sym=None), dict(scale=None), dict(counts=A + 4),
                                dict(sym=None, scale=None, counts=A), dict(sym=None, scale=None, stored=1), dict(yd=3),
                                dict(ldy=63), dict(y=7 * A + 1), dict(rstd=8 * A + 2), dict(res=None, total=4 * A),
                                dict(res=None, total=None, sum_dtype=F32), dict(total=A, lds=128), dict(total=2 * A, lds=65),
                                dict(total=A, sum_dtype=F32)] + [dict(m=m) for m in BAD_MASKS])
def test_norm_refuses(kw):
    assert norm(**kw) == BAD


def test_norm_sizes():
    none = dict(x=None, res=None, w=None, total=None, sym=None, scale=None, y=None, rstd=None)
    assert norm(rows=0, **none) == OK and norm(cols=0, **none) == OK
    assert norm(cols=1 << 31, ld=1 << 31, ldr=1 << 31, lds=1 << 31, ldy=1 << 31) == BIG
    assert norm(rows=1 << 40) == BIG
    for wide in ("ld", "ldr", "lds", "ldy"):
        assert norm(rows=1 << 20, **{wide: 1 << 45}) == BIG


@pytest.mark.parametrize("kw", [dict(dy=None), dict(dy=A + 1), dict(dtype=5), dict(sum_dtype=F16), dict(dtype=F32),
                                dict(ld=63), dict(total=None), dict(total=2 * A + 1), dict(lds=63), dict(q=q8()),
                                dict(total=None, q=q8(rows=3)), dict(total=None, q=q8(cols=32)), dict(total=None, q=q8(fmt=2)),
                                dict(total=None, q=q8(sym=None)), dict(total=None, q=q8(ld=63)), dict(total=None, q=q8(lds=1)),
                                dict(wd=3), dict(w=3 * A + 2), dict(rstd=None), dict(rstd=4 * A + 2), dict(ds=5 * A + 1),
                                dict(ldds=63), dict(ldr=63), dict(dres=6 * A + 1), dict(dx=7 * A + 1), dict(ldx=63),
                                dict(dw=8 * A + 2), dict(dwd=3), dict(dw=3 * A), dict(dres=5 * A, ldr=65),
                                dict(dx=A, ldx=65)] + [dict(m=m) for m in BAD_MASKS])
def test_norm_backward_refuses(kw):
    assert back(**kw) == BAD


def test_norm_backward_sizes():
    # few rows take one launch and no room; more of them, or long ones, need it for partial sums
    assert pc.pc_rmsnorm_backward_workspace_bytes(4, 64) == 0 and pc.pc_rmsnorm_backward_workspace_bytes(512, 8192) == 0
    for rows, cols in ((513, 64), (512, 8200), (4, 8200)):
        need = pc.pc_rmsnorm_backward_workspace_bytes(rows, cols)
        wide = dict(rows=rows, cols=cols, ld=cols, lds=cols, ldds=cols, ldr=cols, ldx=cols)
        assert need > 0 and back(wsb=need - 1, **wide) == SMALL
        assert back(ws=None, **wide) == BAD and back(ws=9 * A + 8, **wide) == BAD
    assert pc.pc_rmsnorm_backward_workspace_bytes(0, 64) == 0 and pc.pc_rmsnorm_backward_workspace_bytes(4, 0) == 0
    assert pc.pc_rmsnorm_backward_workspace_bytes(1 << 40, 64) == 0
    nothing = dict(dy=None, total=None, w=None, rstd=None, ds=None, dres=None, dx=None, ws=None, wsb=0)
    assert back(rows=0, acc=1, **nothing) == OK and back(rows=0, dw=None, **nothing) == OK
    assert back(cols=0, **nothing) == OK
    assert back(cols=1 << 31, ld=1 << 31, lds=1 << 31, ldds=1 << 31, ldr=1 << 31, ldx=1 << 31) == BIG
    assert back(rows=1 << 40) == BIG
    for wide in ("ld", "lds", "ldds", "ldr", "ldx"):
        assert back(rows=1 << 20, **{wide: 1 << 45}) == BIG


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=A + 1), dict(dtype=3), dict(ld=99), dict(vocab=0), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=2.0 ** 65),
                                dict(scale=2.0 ** -65), dict(tok=None), dict(tok=2 * A + 4), dict(tb=2), dict(out=None),
                                dict(out=3 * A + 2), dict(top=101), dict(index=None), dict(index=4 * A + 4), dict(value=None),
                                dict(value=5 * A + 2), dict(stats=6 * A + 2), dict(status=A + 2)])
def test_logprobs_refuses(kw):
    assert logp(**kw) == BAD


def test_logprobs_sizes():
    assert logp(rows=0, x=None, tok=None, out=None, index=None, value=None, stats=None) == OK
    assert logp(m=65) == BIG and logp(vocab=1000, ld=1000, top=65) == BIG
    assert logp(vocab=1 << 31, ld=1 << 31) == BIG and logp(rows=1 << 31) == BIG and logp(rows=1 << 40) == BIG
    assert logp(rows=1 << 20, ld=1 << 45) == BIG
    # few rows of many logits are split: that needs room for the parts
    need = pc.pc_logprobs_workspace_bytes(1, 128000, 20)
    assert need > pc.pc_logprobs_workspace_bytes(1, 128000) > 0
    big = dict(rows=1, vocab=128000, ld=128000, top=20)
    assert logp(wsb=need - 1, **big) == SMALL and logp(ws=None, wsb=0, **big) == BAD
    assert logp(ws=7 * A + 8, wsb=need, **big) == BAD
    assert pc.pc_logprobs_workspace_bytes(4096, 128000) == 0
    for refused in ((0, 100), (1, 0), (1 << 40, 100), (1, 100, 101), (1, 1000, 65), (1, 100, 0, 9)):
        assert pc.pc_logprobs_workspace_bytes(*refused) == 0


@pytest.mark.parametrize("kw", [dict(x=None), dict(dtype=3), dict(ld=99), dict(vocab=0), dict(scale=0.0),
                                dict(scale=math.nan), dict(stats=None), dict(stats=2 * A + 2), dict(tok=None), dict(tb=3),
                                dict(tok=3 * A + 4), dict(d=None), dict(d=4 * A + 2), dict(de=5 * A + 2), dict(out=None),
                                dict(ldo=99), dict(out=6 * A + 1), dict(out=A, ldo=101)])
def test_logprobs_backward_refuses(kw):
    assert logp_back(**kw) == BAD


def test_logprobs_backward_sizes():
    assert logp_back(rows=0, x=None, stats=None, tok=None, d=None, de=None, out=None) == OK
    assert logp_back(m=65) == BIG and logp_back(rows=1 << 31) == BIG
    assert logp_back(rows=1 << 20, ld=1 << 45) == BIG and logp_back(rows=1 << 20, ldo=1 << 45) == BIG


@pytest.mark.parametrize("rows,vocab", [(1 << 31, 1), (1 << 21, 1 << 16), (1, 1 << 31), (1 << 22, 1 << 19)])
def test_logprobs_limits(rows, vocab):
    assert pc.pc_logprobs_workspace_bytes(rows, vocab) == 0
    assert logp(rows=rows, vocab=vocab, ld=vocab, top=0) == BIG
    assert logp_back(rows=rows, vocab=vocab, ld=vocab, ldo=vocab) == BIG


@pytest.mark.parametrize("rows,vocab", [(1, (1 << 31) - 1), (256, 1 << 27), (2, 1 << 30)])
def test_logprobs_just_inside(rows, vocab):
    # recognised by a later refusal (no workspace): no call here reaches the device
    assert pc.pc_logprobs_workspace_bytes(rows, vocab) > 0
    assert logp(rows=rows, vocab=vocab, ld=vocab, top=0, ws=None, wsb=0) == BAD


def test_masks_are_checked():
    for p in (-0.1, 1.5, math.nan):
        with pytest.raises(ValueError):
            pc.DropoutMask(p)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(offset=-1), dict(offset=1 << 64)):
        with pytest.raises(ValueError):
            pc.DropoutMask(0.1, **kw)
    with pytest.raises(TypeError):
        pc.DropoutMask(0.1, 0.5)
    with pytest.raises(TypeError):  # in host memory
        pc.DropoutMask(0.1, torch.zeros(2, dtype=torch.int64))
    m = pc.DropoutMask(0.25, (1 << 64) - 1, 7)
    assert (m.arg.p, m.arg.seed, m.arg.offset, m.arg.d_random) == (0.25, (1 << 64) - 1, 7, None)


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    calls = [lambda: pc.pc_dropout(x, pc.DropoutMask(0.1)), lambda: pc.pc_rmsnorm_store(x),
             lambda: pc.pc_rmsnorm_backward(x, x, None, f), lambda: pc.pc_logprobs(x, t),
             lambda: pc.pc_logprobs_backward(x, torch.zeros(4, 4), t, f)]
    for call in calls:
        with pytest.raises(TypeError, match="device tensor"):
            call()
    for call in (lambda: pc.pc_dropout(x.double(), pc.DropoutMask(0.1)), lambda: pc.pc_rmsnorm_store(x.to(torch.int32)),
                 lambda: pc.pc_logprobs(x.to(torch.int8), t)):
        with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
            call()
    with pytest.raises((TypeError, ValueError)):
        pc.pc_logprobs(x, t, scale="one")
    with pytest.raises(TypeError):
        pc.pc_logprobs(x, t, top=1.5)
    with pytest.raises(TypeError):
        pc.pc_logprobs(x, t, padding=None)
