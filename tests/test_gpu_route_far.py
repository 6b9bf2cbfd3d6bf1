"""The expert router on scores far below binary32's range, against weights formed from log-scores in 64 bits."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import check_close

pytestmark = pytest.mark.gpu


def route(x, k, sigmoid, norm, bias=None, scale=1.0):
    tok, E = x.shape
    xd, b = x.cuda(), bias.cuda() if bias is not None else None
    ids, w = torch.full((tok, k), -7, dtype=torch.int32, device="cuda"), torch.full((tok, k), -7.0, device="cuda")
    code = T.TCM_F32_F32 | (T.TCM_ROUTE_SIGMOID if sigmoid else 0) | (T.TCM_ROUTE_NORM if norm else 0)
    assert T.tcm_moe_route(tok, E, k, xd.data_ptr(), E, code, b.data_ptr() if b is not None else None, scale, ids.data_ptr(), w.data_ptr(),
                           torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    return ids.cpu(), w.cpu()


def check(x, k, sigmoid, norm, bias=None, scale=1.0):
    """ids exactly; weights within the binary32 error of scores down to 2^-100 and of nothing but the result's rounding
    below: arguments up to 70 off by half a step, an exponential, sums over experts and slots, a quotient and a product."""
    ids, w = route(x, k, sigmoid, norm, bias, scale)
    x = x.double()
    log_score = torch.nn.functional.logsigmoid(x) if sigmoid else torch.log_softmax(x, 1)
    key = x if bias is None else log_score.exp() + bias.double()
    rid = torch.argsort(-key, dim=1, stable=True)[:, :k]
    assert torch.equal(ids, rid.to(torch.int32))
    chosen = log_score.gather(1, rid)
    ref = (torch.softmax(chosen, 1) if norm else chosen.exp()) * scale
    rel = 2 * (70 + 16 + x.shape[1] / 64 + k) * 2.0 ** -24
    check_close(w, ref, ref * rel + 2.0 ** -149)


@pytest.mark.parametrize("base", [-60.0, -80.0, -87.0, -88.5, -95.0, -103.0, -110.0, -200.0, -700.0, -720.0, -1000.0, -1e5])
@pytest.mark.parametrize("E,k", [(8, 4), (64, 6), (256, 8), (700, 40)])
def test_sigmoid_of_far_logits(base, E, k):
    gen = torch.Generator().manual_seed(int(-base) + E)
    x = base - 6 * torch.rand(9, E, generator=gen)
    for norm in (True, False):
        check(x, k, True, norm)
        check(x, k, True, norm, bias=torch.randn(E, generator=gen), scale=2.5)


@pytest.mark.parametrize("below", [60.0, 75.0, 88.0, 90.0, 104.0, 110.0, 130.0, 700.0, 760.0, 2000.0])
@pytest.mark.parametrize("E", [12, 100, 300])
def test_softmax_whose_bias_picks_far_experts(below, E):
    gen = torch.Generator().manual_seed(int(below))
    x = -below - 3 * torch.rand(7, E, generator=gen)
    x[:, 5] = 0
    bias = torch.zeros(E)
    bias[[2, 7, 8, 11]] = torch.tensor([2.0, 3.0, 4.0, 5.0])
    for norm in (True, False):
        check(x, 4, False, norm, bias=bias)
        check(x, 5, False, norm, bias=bias)  # (the near one as well)


def test_scores_across_the_subnormal_range():
    x = torch.full((3, 10), -50.0)
    x[:, 0] = 0
    x[0, 1:6] = torch.tensor([-86.0, -88.0, -96.0, -103.5, -120.0])
    x[1, 1:6] = torch.tensor([-103.0, -103.5, -104.0, -105.0, -110.0])
    x[2, 1:6] = torch.tensor([-69.0, -69.5, -70.0, -87.3, -87.4])
    bias = torch.zeros(10)
    bias[1:6] = torch.tensor([2.0, 3.0, 4.0, 5.0, 6.0])
    for norm in (True, False):
        check(x, 5, False, norm, bias=bias)
        check(x[:, 1:], 5, True, norm, bias=bias[1:])


def test_a_large_scale_brings_small_scores_back():
    x = torch.tensor([[-100.0, -101.0, -102.0, -103.0], [-10.0, -95.0, -120.0, -130.0]])
    check(x, 4, True, False, scale=1e30)
    check(x + 10.0, 4, False, False, scale=1e30)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_next_to_far_logits(sigmoid):
    """-inf has a score of zero however small the others are; equal logits of the type's lowest value share the weights."""
    x = torch.full((3, 70), float("-inf"))
    x[0, [3, 66]] = torch.tensor([-95.0, -96.0])
    x[1, 9] = -1e6
    x[2, :] = torch.finfo(torch.float32).min
    ids, w = route(x, 4, sigmoid, True)
    assert torch.equal(ids, torch.tensor([[3, 66, 0, 1], [9, 0, 1, 2], [0, 1, 2, 3]], dtype=torch.int32))
    r = torch.softmax(torch.tensor([-95.0, -96.0], dtype=torch.float64), 0)
    ref = torch.tensor([[r[0], r[1], 0, 0], [1, 0, 0, 0], [0.25] * 4], dtype=torch.float64)
    check_close(w, ref, ref * (2 * (70 + 16 + 2 + 4) * 2.0 ** -24))
