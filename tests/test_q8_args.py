"""Refusals of the stored-tensor and embedding operators, on the CPU: every
call is rejected, or has nothing to do, before the library touches the device
(fake addresses, never dereferenced)."""
import ctypes as C

import pytest
import torch

import static_codebook_lossless_amd as pc
from static_codebook_lossless_amd._lib import StoredArg

lib = pc._lib.lib
P = C.c_void_p
A = 1 << 20
BAD, BIG, SMALL, OK = pc.PC_ERR_INVALID_ARG, pc.PC_ERR_UNSUPPORTED, pc.PC_ERR_CAPACITY, pc.PC_OK


def q8(rows=4, cols=64, sym=A, scale=A, ld=None, lds=None, fmt=0):
    return StoredArg(sym, scale, rows, cols, cols if ld is None else ld, -(-cols // 32) if lds is None else lds, fmt, 0)


def store(x=A, dtype=2, rows=4, cols=64, ld=64, fmt=0, sym=A, scale=A, counts=None):
    return lib.pc_q8_store(x, dtype, rows, cols, ld, fmt, sym, scale, counts, None)


def load(q=None, out=A, dtype=2, ld=64):
    return lib.pc_q8_load(q8() if q is None else q, out, dtype, ld, None)


def glu(dh=A, dtype=2, ld=64, gate=None, up=None, act=0, dg=A * 2, ldg=64, du=A * 3, ldu=64, h=None, ldh=64):
    return lib.pc_q8_glu_backward(dh, dtype, ld, q8() if gate is None else gate, q8() if up is None else up, act, dg,
                                  ldg, du, ldu, h, ldh, None)


def wgrad(dy=A, dtype=2, ld=16, n=16, x=None, dw=A, odt=0, ldw=64, acc=0, ws=A, wsb=1 << 40):
    return lib.pc_q8_weight_grad(dy, dtype, ld, n, q8() if x is None else x, dw, odt, ldw, acc, ws, wsb, None)


def embed(tok=A, tb=8, n=5, table=A, dtype=2, vocab=10, dim=64, ld=64, out=A, odt=2, ldo=64, status=None):
    return lib.pc_embed(tok, tb, n, table, dtype, vocab, dim, ld, 1.0, out, odt, ldo, status, None)


def back(dy=A, dtype=2, ld=64, tok=A, tb=8, n=5, dim=64, vocab=10, grad=A, odt=0, ldg=64, acc=0, ws=A, wsb=1 << 40):
    return lib.pc_embed_backward(dy, dtype, ld, tok, tb, n, dim, vocab, -1, 1.0, grad, odt, ldg, acc, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(sym=None), dict(scale=None), dict(dtype=3), dict(dtype=-1),
                                dict(fmt=2), dict(ld=63), dict(x=A + 1), dict(counts=A + 4)])
def test_store_refuses(kw):
    assert store(**kw) == BAD


def test_store_sizes():
    assert store(cols=1 << 31, ld=1 << 31) == BIG
    assert store(rows=1 << 40) == BIG
    assert store(rows=1 << 20, ld=1 << 45) == BIG
    assert store(rows=0, x=None, sym=None, scale=None) == OK
    assert store(cols=0, x=None, sym=None, scale=None) == OK


@pytest.mark.parametrize("q", [q8(sym=None), q8(scale=None), q8(ld=63), q8(lds=1), q8(fmt=2), q8(fmt=-1)])
def test_stored_tensors_are_checked(q):
    assert load(q) == BAD
    assert glu(gate=q) == BAD
    assert glu(up=q) == BAD
    assert wgrad(x=q) == BAD
    assert lib.pc_embed_q8(A, 8, 5, q, 1.0, A, 2, 64, None, None) == BAD


def test_load_refuses():
    assert load(out=None) == BAD and load(dtype=7) == BAD and load(ld=63) == BAD and load(out=A + 1) == BAD
    assert load(out=A + 2, dtype=0) == BAD
    assert lib.pc_q8_load(None, A, 2, 64, None) == BAD
    assert load(q8(rows=0, sym=None, scale=None), out=None) == OK
    assert load(q8(rows=1 << 40)) == BIG


@pytest.mark.parametrize("kw", [dict(dh=None), dict(dtype=5), dict(act=3), dict(act=-1), dict(dg=None), dict(du=None),
                                dict(ld=10), dict(ldg=10), dict(ldu=10), dict(h=A, ldh=10), dict(up=q8(rows=3)),
                                dict(up=q8(cols=32)), dict(up=q8(fmt=1)), dict(dg=A, ldg=128)])
def test_glu_refuses(kw):
    assert glu(**kw) == BAD


def test_glu_without_gate_has_no_second_gradient():
    assert lib.pc_q8_glu_backward(A, 2, 64, q8(), None, 0, A, 64, A, 64, None, 0, None) == BAD
    assert lib.pc_q8_glu_backward(None, 2, 64, q8(rows=0), None, 0, None, 64, None, 64, None, 0, None) == OK


@pytest.mark.parametrize("kw", [dict(dy=None), dict(dtype=3), dict(odt=3), dict(dw=None), dict(ld=15), dict(ldw=63),
                                dict(dy=A + 1), dict(dw=A + 2)])
def test_weight_grad_refuses(kw):
    assert wgrad(**kw) == BAD


def test_weight_grad_workspace():
    need = pc.pc_q8_weight_grad_workspace_bytes(65536, 64, 64)
    assert need > 0
    x = q8(rows=65536)
    assert wgrad(x=x, n=64, ld=64, wsb=need - 1) == SMALL
    assert wgrad(x=x, n=64, ld=64, ws=None, wsb=0) == BAD
    assert wgrad(x=x, n=64, ld=64, ws=A + 8, wsb=need) == BAD
    assert pc.pc_q8_weight_grad_workspace_bytes(0, 64, 64) == 0
    assert wgrad(n=0, dw=None) == OK
    assert wgrad(x=q8(rows=0), acc=1) == OK
    assert wgrad(n=1 << 31, ld=1 << 31) == BIG
    assert wgrad(ld=1 << 24) == BIG and wgrad(x=q8(ld=1 << 24)) == BIG and wgrad(x=q8(lds=1 << 24)) == BIG


@pytest.mark.parametrize("kw", [dict(tok=None), dict(tb=2), dict(tok=A + 4), dict(table=None), dict(dtype=9),
                                dict(odt=9), dict(ld=63), dict(ldo=63), dict(out=None), dict(status=A + 1)])
def test_embed_refuses(kw):
    assert embed(**kw) == BAD


def test_embed_sizes():
    assert embed(n=0, tok=None, table=None, out=None) == OK
    assert embed(dim=0, tok=None, table=None, out=None) == OK
    assert embed(n=1 << 45) == BIG
    assert lib.pc_embed_q8(A, 8, 5, None, 1.0, A, 2, 64, None, None) == BAD


@pytest.mark.parametrize("kw", [dict(dy=None), dict(tok=None), dict(tb=3), dict(tok=A + 4), dict(dtype=9), dict(odt=9),
                                dict(ld=63), dict(ldg=63), dict(grad=None), dict(n=5000, ws=None), dict(n=5000, ws=A + 8)])
def test_embed_backward_refuses(kw):
    assert back(**kw) == BAD


def test_embed_backward_sizes():
    need = pc.pc_embed_backward_workspace_bytes(5000, 64, 10)
    assert back(n=5000, wsb=need - 1) == SMALL
    assert back(n=1 << 31) == BIG and back(vocab=(1 << 31) + 1) == BIG
    assert back(n=0, acc=1, dy=None, tok=None) == OK
    assert back(vocab=0, grad=None) == OK and back(dim=0, grad=None) == OK
    assert pc.pc_embed_backward_workspace_bytes(1 << 31, 64, 10) == 0


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    s, c = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        pc.pc_q8_store(x)  # host memory
    with pytest.raises(ValueError):
        pc.pc_q8_store(x, "e5m2")
    with pytest.raises(TypeError):
        pc.pc_q8_store(x.double())
    with pytest.raises(TypeError):
        pc.Q8(s, c)
    with pytest.raises(TypeError):
        pc.Q8(s.float(), c)
    with pytest.raises(ValueError):
        pc.Q8(s, c, "int4")
    with pytest.raises(ValueError):
        pc.Q8(s[0], c)
    with pytest.raises(TypeError):
        pc.pc_embed(torch.zeros(3, dtype=torch.int64), x)
    with pytest.raises(TypeError):
        pc.pc_embed_q8(torch.zeros(3, dtype=torch.int64), x)
    with pytest.raises(ValueError):
        pc.pc_embed_backward(x, torch.zeros(3, dtype=torch.int64), 10)
