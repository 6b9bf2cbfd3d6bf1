"""An expert layer whose tokens x hidden passes what one launch of its sum takes."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import check_close, half_step, moe_ref

pytestmark = pytest.mark.gpu


def test_wide_rows_of_many_tokens():
    tok, H, I = 1024, 1 << 22, 2  # 2^32 outputs
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = torch.empty(tok, H, dtype=torch.bfloat16, device="cuda")
    for t in range(0, tok, 128):
        x[t:t + 128] = rnd(128, H).bfloat16()
    w1, w2 = (rnd(1, 2, I, H) * H ** -0.5).bfloat16(), (rnd(1, H, I) * I ** -0.5).bfloat16()
    ids, wt = torch.zeros(tok, 1, dtype=torch.int32, device="cuda"), torch.rand(tok, 1, generator=gen, device="cuda")
    out = torch.full((tok, H), 7.0, dtype=torch.bfloat16, device="cuda")
    assert T.tcm_moe(tok, H, I, 1, 1, x.data_ptr(), H, ids.data_ptr(), wt.data_ptr(), w1.data_ptr(), None, w2.data_ptr(), None,
                     out.data_ptr(), H, T.TCM_BF16_F32 | T.TCM_C_BF16, torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    assert "moe_tile" in T.tcm_last_plan()
    at = [0, 511, 1022, 1023]
    ref, bound = moe_ref(x[at].cpu(), ids[at].cpu(), wt[at].cpu(), w1.cpu(), None, w2.cpu(), None)
    check_close(out[at].cpu(), ref, bound + half_step(ref, torch.bfloat16) * (1 + 2.0 ** -10) + 2.0 ** -126)
    assert not (out[:, ::65537] == 7).all(1).any()  # every token was written
    T.tcm_release_workspace()  # (17 GB of it)
