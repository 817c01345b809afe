"""Outputs of the norm's backward pass in an input's place: those that the header
allows are accepted, the others refused (on the CPU, by addresses that are never
dereferenced)."""
import itertools

import pytest

from test_step_args import A, BAD, BF16, F32, SMALL, back, mask, q8

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
