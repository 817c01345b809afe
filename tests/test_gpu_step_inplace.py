"""Tensors whose memory changes between calls."""
import pytest
import torch

from test_gpu_step import DEV

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
