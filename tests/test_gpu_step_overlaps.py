"""The norm's gradients in the place of its inputs, in every pairing that the header allows."""
import itertools

import numpy as np
import pytest
import torch

from test_gpu_step import DEV, DT, activation, say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import static_codebook_lossless_amd as pc


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# one launch (up to 512 rows), two, ragged ones, long rows
@pytest.mark.parametrize("rows,cols", [(70, 264), (512, 8192), (400, 5001), (600, 520), (5, 8191), (3, 40001), (600, 16400)])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f16", "f32")])
def test_gradients_over_inputs(rows, cols, dtype, res):
    lib, kinds = pc._lib.lib, {"f32": pc.PC_F32, "f16": pc.PC_F16, "bf16": pc.PC_BF16}
    rng = np.random.default_rng(81)
    given = [activation(rng, rows, cols, dtype), activation(rng, rows, cols, res), activation(rng, rows, cols, res)]
    w, rstd = torch.rand(cols, device=DEV), torch.rand(rows, device=DEV)
    mask = pc.DropoutMask(0.3, 4)
    want = pc.pc_rmsnorm_backward(given[0], given[1], w, rstd, d_sum=given[2], mask=mask)
    need = pc.pc_rmsnorm_backward_workspace_bytes(rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for a, b in itertools.product((None, 0, 1, 2), repeat=2):
        if a == b or (a == 0 and dtype != res) or (b in (1, 2) and dtype != res):
            continue
        say("overlap", rows, cols, dtype, res, a, b)
        dy, h, ds = (t.clone() for t in given)
        d_res = torch.empty(rows, cols, dtype=DT[res], device=DEV) if a is None else (dy, h, ds)[a]
        d_x = torch.empty(rows, cols, dtype=DT[dtype], device=DEV) if b is None else (dy, h, ds)[b]
        dw = torch.empty(cols, device=DEV)
        st = lib.pc_rmsnorm_backward(dy.data_ptr(), kinds[dtype], rows, cols, cols, h.data_ptr(), kinds[res], cols, None,
                                     w.data_ptr(), pc.PC_F32, rstd.data_ptr(), ds.data_ptr(), cols, mask.arg,
                                     d_res.data_ptr(), cols, d_x.data_ptr(), cols, dw.data_ptr(), pc.PC_F32, 0,
                                     ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == pc.PC_OK
        assert torch.equal(d_res, want.residual) and torch.equal(d_x, want.x) and torch.equal(dw, want.weight)


@pytest.mark.parametrize("rows,cols", [(70, 264), (300, 96), (9, 8192), (3, 16390), (3, 40001)])
@pytest.mark.parametrize("with_sum", [True, False])
def test_y_over_inputs(rows, cols, with_sum):
    lib = pc._lib.lib
    rng = np.random.default_rng(82)
    given = [activation(rng, rows, cols, "bf16") for _ in range(2)]
    mask = pc.DropoutMask(0.3, 4)
    want = pc.pc_rmsnorm_store(given[0], None, given[1], mask, y="plain")
    for k in range(2):
        x, res = (t.clone() for t in given)
        y, total = (x, res)[k], torch.empty_like(x) if with_sum else None
        st = lib.pc_rmsnorm_store(x.data_ptr(), pc.PC_BF16, rows, cols, cols, res.data_ptr(), pc.PC_BF16, cols, mask.arg,
                                  None, 0, 1e-6, None if total is None else total.data_ptr(), cols, 0, None, None, None,
                                  y.data_ptr(), pc.PC_BF16, cols, 0, None, torch.cuda.current_stream().cuda_stream)
        assert st == pc.PC_OK and torch.equal(y, want.y) and (total is None or torch.equal(total, want.sum))
