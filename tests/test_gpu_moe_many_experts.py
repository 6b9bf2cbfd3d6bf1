"""Experts whose doubled number passes 31 bits (the two matrices of each lie one after the other)."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import check_close, half_step, moe_ref

pytestmark = pytest.mark.gpu


def test_experts_past_2_30():
    E, H, I, tok = (1 << 30) + 3, 1, 1, 4  # one weight a matrix
    far = [5, (1 << 29) + 1, 1 << 30, E - 1]
    gen = torch.Generator().manual_seed(0)
    w1, w2 = torch.randn(4, 2, I, H, generator=gen).half(), torch.randn(4, H, I, generator=gen).half()
    W1, W2 = torch.zeros(E, 2, I, H, dtype=torch.float16, device="cuda"), torch.zeros(E, H, I, dtype=torch.float16, device="cuda")
    for j, e in enumerate(far):
        W1[e], W2[e] = w1[j].cuda(), w2[j].cuda()
    x, wt = torch.randn(tok, H, generator=gen).half(), torch.rand(tok, 2, generator=gen)
    ids = torch.tensor([[0, 3], [2, 1], [3, 2], [1, 0]], dtype=torch.int32)
    idd, xd, wd = torch.tensor(far, dtype=torch.int32)[ids.long()].cuda(), x.cuda(), wt.cuda()
    out = torch.full((tok, H), 7.0, dtype=torch.float16, device="cuda")
    assert T.tcm_moe(tok, H, I, E, 2, xd.data_ptr(), H, idd.data_ptr(), wd.data_ptr(), W1.data_ptr(), None, W2.data_ptr(), None,
                     out.data_ptr(), H, T.TCM_F16_F32 | T.TCM_C_F16, torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    assert "moe_generic" in T.tcm_last_plan()
    ref, bound = moe_ref(x, ids, wt, w1, None, w2, None)
    check_close(out.cpu(), ref, bound + half_step(ref, torch.float16) * (1 + 2.0 ** -10) + 2.0 ** -126)
