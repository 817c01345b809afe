"""The binding of the norm, dropout and log-probability operators, on the CPU: numbers that an argument's type
cannot hold, and what a mask was made of."""
import pytest
import torch

import static_codebook_lossless_amd as pc


@pytest.mark.parametrize("padding", [1 << 63, -(1 << 63) - 1, 1 << 64, (1 << 64) + 5])
def test_padding_of_more_than_64_bits(padding):
    """Taken modulo 2^64, it would be another token."""
    x, t = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="64 bits"):
        pc.pc_logprobs(x, t, padding=padding)
    with pytest.raises(ValueError, match="64 bits"):
        pc.pc_logprobs_backward(x, torch.zeros(4, 4), t, torch.zeros(4), padding=padding)


@pytest.mark.parametrize("padding", [(1 << 63) - 1, -(1 << 63), -1, 0])
def test_padding_of_64_bits(padding):
    with pytest.raises(TypeError, match="device tensor"):  # the next check
        pc.pc_logprobs(torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64), padding=padding)


def test_a_mask_stays_what_it_was_made_of():
    """What its argument was made from cannot be set to something else beside it."""
    m = pc.DropoutMask(0.25, 5, 6)
    for name, value in (("p", 0.5), ("seed", 7), ("offset", 8)):
        with pytest.raises(AttributeError):
            setattr(m, name, value)
    assert (m.p, m.seed, m.offset) == (0.25, 5, 6) and (m.arg.p, m.arg.seed, m.arg.offset) == (0.25, 5, 6)
