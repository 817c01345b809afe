"""The order in which log probabilities are summed: by sizes alone."""
import pytest
import torch

from test_gpu_step import DEV, DT, say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 1, 5600000), ("bf16", 2, 2000000), ("f32", 1, 400001),
                                              ("f16", 5, 420000), ("f32", 7, 150000)])
def test_alternatives_change_no_sum(dtype, rows, vocab):
    """Sums of splits are added in one order, with alternatives or without."""
    g = torch.Generator(device=DEV).manual_seed(7)
    for k in range(12):
        say("order", dtype, rows, vocab, k)
        x = (torch.randn(rows, vocab, generator=g, device=DEV) * (0.5 + k)).to(DT[dtype])
        tokens = torch.randint(0, vocab, (rows, 3), generator=g, device=DEV)
        a, b = pc.pc_logprobs(x, tokens), pc.pc_logprobs(x, tokens, top=6)
        assert torch.equal(a.stats, b.stats) and torch.equal(a.logp, b.logp), k
