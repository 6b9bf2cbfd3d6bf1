"""Losses far below 1: choices that the scores hardly favour, and logs of sums next to 1."""
import math

import pytest
import torch

import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 100, 128, 129, 3000])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("far", [2.0, 12.0, 17.0, 30.0])
def test_all_choices_on_a_small_share(tokens, far, sigmoid):
    """All choices on an expert whose logit lies far / 2 below most and 1.5 far below another.  Up to 128 tokens to the
    reference's bound, which is relative; with more the sum's 2^-34 besides, less than a thousandth of the loss up to 12."""
    E = 1024
    x = torch.full((tokens, E), 0.0)
    x[:, 3] = far
    x[:, 5] = -far / 2
    ids = torch.full((tokens, 1), 5, dtype=torch.int32)
    counts, losses = R.run_balance(x, ids, None, sigmoid)
    want, ref, bound = R.loss_ref(x, ids, None, sigmoid)
    assert torch.equal(counts, want)
    assert float(bound[0]) < 1e-4 * float(ref[0]) and (far > 12 or 2.0 ** -34 < 1e-3 * float(ref[0]))
    assert abs(float(losses[0]) - float(ref[0])) <= float(bound[0]) + (2.0 ** -34 if tokens > 128 else 0.0)
    assert float(losses[0]) > 0 or (tokens > 128 and float(ref[0]) < 2.0 ** -34)


@pytest.mark.parametrize("tokens", [1, 100, 3000])
@pytest.mark.parametrize("E,x", [(1, 1e-4), (1, -3e-6), (2, -math.log(2.0)), (300, -math.log(300.0) + 1e-3), (5, 0.0)])
def test_logs_next_to_zero(tokens, E, x):
    """The reference's bound: steps of the logits and of the sum, not of the log itself."""
    counts, losses = R.run_balance(torch.full((tokens, E), x), torch.zeros(tokens, 1, dtype=torch.int32), None, False)
    want, ref, bound = R.loss_ref(torch.full((tokens, E), x), torch.zeros(tokens, 1, dtype=torch.int32), None, False)
    assert torch.equal(counts, want) and ((losses.double() - ref).abs() <= bound + (2.0 ** -34 if tokens > 128 else 0.0)).all()
    assert (losses[1] >= 0).all()
