"""The size limits of the stored-tensor and embedding operators, on the CPU,
just inside and just outside.  A size inside is recognised by a later refusal
(no workspace): no call here reaches the device."""
import pytest
import torch

import static_codebook_lossless_amd as pc
from test_q8_args import A, BAD, BIG, back, q8, wgrad

MI = 1 << 20


@pytest.mark.parametrize("n,dim,vocab", [
    (512 * MI, 1, 10), (512 * MI, 96, 10), (5, 1, 64 * MI - 5), (256 * MI, 1, 56 * MI - 4), (0, 1, 64 * MI - 4),
    (128 * MI - 8, 512, 10), (3000, 1 << 24, 10), (600, 1 << 26, 3)])
def test_embed_backward_accepts(n, dim, vocab):
    assert pc.pc_embed_backward_workspace_bytes(n, dim, vocab) > 0
    assert back(n=n, dim=dim, vocab=vocab, ld=dim, ldg=dim, ws=None, wsb=0) == BAD
    assert back(n=n, dim=dim, vocab=vocab, ld=dim, ldg=dim, ws=A, wsb=16) == pc.PC_ERR_CAPACITY


@pytest.mark.parametrize("n,dim,vocab", [
    (512 * MI + 1, 1, 10), (5, 1, 64 * MI - 4), (256 * MI, 1, 56 * MI - 3), (0, 1, 64 * MI - 3), (128 * MI, 512, 10),
    (512 * MI, 128, 10), (5, 1 << 16, 1 << 20), (1 << 31, 64, 10)])
def test_embed_backward_refuses_what_it_cannot_launch(n, dim, vocab):
    assert pc.pc_embed_backward_workspace_bytes(n, dim, vocab) == 0
    assert back(n=n, dim=dim, vocab=vocab, ld=dim, ldg=dim) == BIG


@pytest.mark.parametrize("n,k", [(1, (1 << 31) - 1), ((1 << 31) - 128, 1)])
def test_weight_grad_of_no_rows_refuses_what_it_cannot_launch(n, k):
    # 2^24 tiles of 256 lanes: no launch holds them, also where they only write zeros
    assert wgrad(x=q8(rows=0, cols=k), dtype=pc.PC_F32, n=n, ld=n, ldw=k) == BIG


def test_binding_raises_type_and_value_errors():
    s, c = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    q = pc.Q8._dense(s, c, "e4m3", 4, 64, 0)  # in host memory, where only the checks are reached
    with pytest.raises(ValueError):
        q.with_symbols(torch.zeros(255, dtype=torch.uint8))
    with pytest.raises(ValueError):
        q.with_symbols(torch.zeros(8, 64, dtype=torch.uint8)[::2].t())
    x = torch.zeros(4, 64)
    for call in (lambda: pc.pc_q8_load(x), lambda: pc.pc_q8_glu_backward(x, x), lambda: pc.pc_q8_glu_backward(x, q, x),
                 lambda: pc.pc_q8_weight_grad(x, x), lambda: pc.pc_embed_q8(torch.zeros(3, dtype=torch.int64), x)):
        with pytest.raises(TypeError, match="must be a Q8"):
            call()
    tokens = torch.zeros(4, dtype=torch.int64)
    with pytest.raises((TypeError, ValueError)):
        pc.pc_embed(tokens, x, scale="two")
    with pytest.raises(TypeError):
        pc.pc_embed_backward(x, tokens, 10, padding=None)
