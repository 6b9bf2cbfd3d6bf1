"""More tokens than one launch of the router takes."""
import pytest
import torch

import tensor_core_mixed_amd as T

pytestmark = pytest.mark.gpu


def test_tokens_past_one_launch():
    tok, E, k = (1 << 26) + 5, 4, 2
    x = torch.zeros(tok, E, dtype=torch.float16, device="cuda")
    band = 1 << 25
    at = torch.cat([torch.arange(c - 7, min(c + 7, tok)) for c in (7, band, 2 * band)]).cuda()  # (the last are the last tokens)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x[at] = torch.randn(len(at), E, generator=gen, device="cuda").half()
    ids, w = torch.full((tok, k), -7, dtype=torch.int32, device="cuda"), torch.full((tok, k), -7.0, device="cuda")
    assert T.tcm_moe_route(tok, E, k, x.data_ptr(), E, T.TCM_F16_F32, None, 1.0, ids.data_ptr(), w.data_ptr(),
                           torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    score = torch.softmax(x[at].double(), 1)
    rid = torch.argsort(-x[at].double(), dim=1, stable=True)[:, :k]
    assert torch.equal(ids[at].long(), rid)
    assert ((w[at].double() - score.gather(1, rid)).abs() <= score.gather(1, rid) * 2.0 ** -18).all()
    zero = torch.ones(tok, dtype=torch.bool, device="cuda")
    zero[at] = False
    assert (ids[zero] == torch.arange(k, device="cuda")).all() and (w[zero] == 0.25).all()
