"""The update's largest tile, in one range of k and in several, for each of a step's three products: sizes that the planner
gives it, with tiles past every edge, tall and wide."""
import pytest
import torch

import tensor_core_mixed_amd as T
from test_gpu_ortho import MUON, check, update

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,rows,cols,plan", [
    # the tiles and the ranges of S, T and X
    (8, 768, 2048, "tile=1,1,0 split=10101"), (8, 2048, 768, "tile=1,1,0 split=10101"), (7, 769, 2049, "tile=1,1,0 split=10101"),
    (2, 2047, 2051, "tile=0,0,0 split=30301"), (3, 2049, 1537, "tile=0,0,0 split=30301"), (8, 1025, 1024, "tile=0,0,0 split=30301"),
    (1, 1281, 20001, "tile=0,2,0 split=120101"), (1, 2500, 2501, "tile=1,1,0 split=10102"), (1, 3334, 3333, "tile=0,0,0 split=20201"),
    (1, 5001, 5003, "tile=0,0,0 split=10101"),
])
def test_largest_tile(batch, rows, cols, plan):
    t = torch.bfloat16 if rows % 2 else torch.float32
    g = update(torch.Generator().manual_seed(rows), batch, rows, cols, t)
    check(g, coef=MUON * 2, out=torch.float32 if rows % 3 else t, pad=rows % 2)
    assert T.tcm_last_plan().endswith(plan), T.tcm_last_plan()


@pytest.mark.parametrize("shape", [(1, 2047, 2051), (1, 4096, 1024), (8, 1025, 1024)])
def test_the_same_bits_again(shape):
    """Whatever ran before it in the workspace."""
    g = update(torch.Generator().manual_seed(1), *shape, torch.bfloat16).cuda()
    b, r, c = shape
    other = torch.randn(1, 1500, 1700, device="cuda")
    junk = torch.empty_like(other)

    def call(x, o, code):
        b, r, c = x.shape
        assert T.tcm_orthogonalize(b, r, c, x.data_ptr(), c, r * c, o.data_ptr(), c, r * c, code, MUON * 5, 1e-7, 1.0,
                                   torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    want = torch.empty_like(g)
    call(g, want, T.TCM_BF16_F32 | T.TCM_C_BF16)
    for turn in range(12):
        o = torch.full_like(g, 9)
        if turn % 3 == 2:
            call(other, junk, T.TCM_F32_F32)
        call(g, o, T.TCM_BF16_F32 | T.TCM_C_BF16)
        torch.cuda.synchronize()
        assert torch.equal(o, want), turn
