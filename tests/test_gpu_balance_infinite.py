"""Logits that are +inf or NaN in the router's losses and gradient, in every form of the scores and weights."""
import math

import pytest
import torch

import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("tokens", [3, 300])
@pytest.mark.parametrize("E", [20, 300])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_losses(bad, tokens, E, sigmoid):
    x, ids, _ = R.inputs(tokens, E, 2, torch.float32)
    clean = R.run_balance(x, ids, None, sigmoid)
    x[1, 3] = bad
    counts, losses = R.run_balance(x, ids, None, sigmoid)
    assert torch.equal(counts, clean[0]) and clean[1].isfinite().all() and losses.isnan().all()
    mask = torch.ones(tokens, dtype=torch.uint8)
    mask[1] = 0
    assert R.run_balance(x, ids, mask, sigmoid)[1].isfinite().all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("E", [20, 300])
@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("weights,losses", [(True, True), (True, False), (False, True)])
def test_gradient(bad, E, sigmoid, norm, weights, losses):
    x, ids, _ = R.inputs(9, E, 2, torch.float32)
    counts, _ = R.run_balance(x, ids, None, sigmoid)
    x[1, 3] = bad
    d = R.run_grad(x, ids, None, sigmoid, norm, torch.randn(9, 2) if weights else None, counts if losses else None,
                   torch.ones(2) if losses else None, 1.0, torch.float32)
    assert d[1].isnan().all() and d[0].isfinite().all() and d[2:].isfinite().all()
