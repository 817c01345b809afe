"""Outputs of the norm and of the logits' gradient in an input's place: those that the header
allows are accepted, the others refused (on the CPU, by addresses that are never
dereferenced)."""
import itertools

import pytest

from test_step_args import A, BAD, BF16, BIG, F32, SMALL, back, logp_back, mask, norm, q8

IN = {"dy": A, "total": 2 * A, "w": 3 * A, "rstd": 4 * A, "ds": 5 * A}
ROWS = ("dy", "total", "ds")

# an accepted call is recognised by a later refusal, a workspace that is too small: none reaches the device
WIDE = dict(rows=600, cols=64, ws=9 * A, wsb=1)


def test_calls_of_their_own_memory_pass():
    assert back(**WIDE) == SMALL


@pytest.mark.parametrize("out,ld", [("dres", "ldr"), ("dx", "ldx")])
@pytest.mark.parametrize("what", ROWS)
def test_rows_in_place(out, ld, what):
    assert back(**{out: IN[what]}, **WIDE) == SMALL
    assert back(**{out: IN[what], ld: 65}, **WIDE) == BAD  # another row distance
    # another type: x's and y's gradients in 16 bits, the sum's in 32
    same = (out == "dx") == (what == "dy")
    assert back(**{out: IN[what]}, dtype=BF16, sum_dtype=F32, **WIDE) == (SMALL if same else BAD)


@pytest.mark.parametrize("out", ["dres", "dx", "dw"])
@pytest.mark.parametrize("what", ["w", "rstd"])
def test_no_output_over_weights_or_roots(out, what):
    assert back(**{out: IN[what]}, **WIDE) == BAD


@pytest.mark.parametrize("out", ["dres", "dx", "dw"])
@pytest.mark.parametrize("what", ["sym", "scale"])
def test_no_output_over_the_stored_sum(out, what):
    at = {"sym": 20 * A, "scale": 21 * A}
    q = q8(rows=600, **at)
    assert back(total=None, q=q, **WIDE) == SMALL
    assert back(total=None, q=q, **{out: at[what]}, **WIDE) == BAD


@pytest.mark.parametrize("what", ROWS)
def test_no_weight_gradient_over_rows(what):
    assert back(dw=IN[what], **WIDE) == BAD


def test_no_two_outputs_in_one_place():
    assert back(dres=7 * A, m=mask(), **WIDE) == BAD
    assert back(dres=7 * A, sum_dtype=F32, **WIDE) == BAD
    assert back(dres=7 * A, ldr=65, **WIDE) == BAD
    assert back(dres=8 * A, **WIDE) == BAD and back(dx=8 * A, **WIDE) == BAD


@pytest.mark.parametrize("a,b", itertools.permutations(ROWS, 2))
def test_both_in_place(a, b):
    assert back(dres=IN[a], dx=IN[b], **WIDE) == SMALL
    assert back(dres=IN[a], dx=IN[a], m=mask(), **WIDE) == BAD


# the forward pass and the logits' gradient: accepted calls are recognised by an alignment that is refused later,
# or by a row distance that is too large

FAR = dict(rows=1 << 20, ld=1 << 45)


def test_y_in_place():
    far = dict(rows=1 << 20, ld=1 << 45, ldr=1 << 45, ldy=1 << 45, lds=64)
    assert norm(**far) == BIG and norm(y=A, **far) == BIG and norm(y=2 * A, **far) == BIG
    assert norm(y=A, **{**far, "ldy": 64}) == BAD and norm(y=2 * A, **{**far, "ldy": 64}) == BAD
    assert norm(y=A, yd=F32, **far) == BAD and norm(y=2 * A, sum_dtype=F32, **far) == BAD
    assert norm(y=4 * A, **{**far, "ldy": 64}) == BAD  # the sum's place


@pytest.mark.parametrize("kw", [dict(sym=A), dict(scale=2 * A), dict(rstd=A), dict(sym=3 * A), dict(rstd=4 * A), dict(rstd=7 * A),
                                dict(scale=5 * A), dict(rstd=5 * A), dict(rstd=6 * A), dict(counts=5 * A), dict(total=3 * A),
                                dict(y=3 * A)])
def test_norm_outputs_of_their_own(kw):
    assert norm(**FAR) == BIG and norm(**kw, **FAR) == BAD


@pytest.mark.parametrize("out", [2, 3, 4, 5])
def test_no_logits_gradient_over_its_other_inputs(out):
    assert logp_back(out=A, ldo=1 << 45, **FAR) == BIG and logp_back(out=6 * A, **FAR) == BIG
    assert logp_back(out=out * A, **FAR) == BAD
