"""The router's losses over many tokens, for one-sided routings, and for logits that are not finite."""
import math

import pytest
import torch

import tensor_core_mixed_amd as T
import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("tokens,E", [((1 << 24) - 5, 3), ((1 << 21) + 1, 257), ((1 << 22) + 77, 60)])
def test_equal_shares_of_many_tokens(tokens, E, sigmoid):
    """Every share is 1 / E: roundings of a long binary32 sum would all go one way.  To 2^-19: a share's own roundings (an
    exponential to two steps of 2^-23, a sigmoid and its inverse, a sum of up to 22 additions and a division: 32 half steps),
    and runs of 16 of them."""
    x = torch.zeros(tokens, E, dtype=torch.float16, device="cuda")
    ids = (torch.arange(tokens, device="cuda") % E).int()
    counts, losses = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    assert T.tcm_moe_balance(tokens, E, 1, x.data_ptr(), E, T.TCM_F16_F32 | (T.TCM_ROUTE_SIGMOID if sigmoid else 0), ids.data_ptr(), None,
                             counts.data_ptr(), losses.data_ptr(), R.stream()) == T.TCM_OK
    torch.cuda.synchronize()
    assert int(counts[-1]) == tokens and int(counts[:-1].sum()) == tokens
    z = math.log(E) ** 2
    assert abs(float(losses[0]) - 1) <= 2.0 ** -19 and abs(float(losses[1]) - z) <= 2.0 ** -20 * z
