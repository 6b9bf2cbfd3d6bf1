"""A token's gradient has the same bits wherever the token lies and whatever the others hold."""
import pytest
import torch

import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(6, 2), (64, 6), (256, 8), (300, 4)])
@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("t", list(R.TYPES))
def test_far_neighbours(E, k, sigmoid, norm, t):
    tokens = 41
    x, ids, _ = R.inputs(tokens, E, k, t)
    gen = torch.Generator().manual_seed(1)
    dw, dl = torch.randn(tokens, k, generator=gen), torch.tensor([3.0, -2.0])
    counts, _ = R.run_balance(x, ids, None, sigmoid)
    near = R.run_grad(x, ids, None, sigmoid, norm, dw, counts, dl, 1.0, torch.float32)
    y = x.clone()
    moved = torch.arange(tokens) % 3 == 0
    y[moved] += 300
    y[0::6] -= 600  # (to -300: sigmoids that binary32 does not hold)
    y[0::9, 1] = -torch.inf
    far = R.run_grad(y, ids, None, sigmoid, norm, dw, counts, dl, 1.0, torch.float32)
    assert torch.equal(far[~moved], near[~moved])
    order = torch.randperm(tokens, generator=gen)
    again = R.run_grad(y[order], ids[order], None, sigmoid, norm, dw[order], counts, dl, 1.0, torch.float32)
    assert torch.equal(again, far[order])
