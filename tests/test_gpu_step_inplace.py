"""Tensors whose memory or contents change between calls, and who hears of it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from test_gpu_step import DEV, activation

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_mask_reads_the_seed_where_it_is():
    """A seed tensor whose memory is replaced (as ``.data`` and ``set_`` do) after the mask was made."""
    x = torch.ones(64, 256, device=DEV)
    seed = torch.tensor([5, 6], device=DEV)
    old = seed.detach()  # keeps the first memory
    mask = pc.DropoutMask(0.5, seed, 3)
    first = pc.pc_dropout(x, mask)
    seed.set_(torch.tensor([7, 9], device=DEV))
    assert old.tolist() == [5, 6] and seed.tolist() == [7, 9]
    assert torch.equal(pc.pc_dropout(x, mask), pc.pc_dropout(x, pc.DropoutMask(0.5, 7, 12)))
    assert torch.equal(first, pc.pc_dropout(x, pc.DropoutMask(0.5, 5, 9)))
    n = pc.pc_rmsnorm_store(x, mask=mask, format=None)
    assert torch.equal(n.sum, pc.pc_dropout(x, pc.DropoutMask(0.5, 7, 12)))


def test_mask_refuses_a_seed_that_no_longer_fits():
    x = torch.ones(4, 64, device=DEV)
    for other in (torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)[::2]):
        seed = torch.tensor([5, 6], device=DEV)
        mask = pc.DropoutMask(0.5, seed)
        seed.set_(other)
        with pytest.raises(TypeError):
            pc.pc_dropout(x, mask)


def writes():
    """(what is written, a call that writes it) for every output that a caller gives."""
    rng = np.random.default_rng(71)
    x = activation(rng, 6, 64, "f32")
    w, rstd, mask = torch.rand(64, device=DEV), torch.rand(6, device=DEV), pc.DropoutMask(0.5, 1)
    tokens = torch.arange(6, device=DEV)
    stats = pc.pc_logprobs(x, tokens).stats
    d = torch.ones(6, device=DEV)
    return [
        (x, lambda out: pc.pc_dropout(x, mask, out=out)),
        (x, lambda out: pc.pc_rmsnorm_store(x, w, residual=x, sum_out=out)),
        (x, lambda out: pc.pc_logprobs_backward(x, stats, tokens, d, out=out)),
        (torch.zeros(64, device=DEV), lambda out: pc.pc_rmsnorm_backward(x, x, w, rstd, weight_out=out)),
        (torch.zeros(64, device=DEV), lambda out: pc.pc_rmsnorm_backward(x, x, w, rstd, weight_out=out, accumulate=True)),
    ]


@pytest.mark.parametrize("k", range(5))
def test_writes_are_seen_by_autograd(k):
    """A tensor that a graph has saved and a call has written since is reported, not used."""
    like, call = writes()[k]
    out = (like.clone().requires_grad_() * 1.0)
    loss = out.square().sum()  # saves out
    call(out.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # in inference mode nothing is counted, and the calls work
    with torch.inference_mode():
        call(like.clone())


def test_example_reports_a_second_backward_pass():
    spec = importlib.util.spec_from_file_location("residual_step", os.path.join(ROOT, "examples", "residual_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model(vocab=64, dim=32, hidden=32)
    tokens = torch.arange(64, device=DEV)
    loss = model.loss(tokens, tokens, torch.ones(64, device=DEV))
    loss.backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
