"""Steps whose polynomial has a fifth power next to nothing: its largest value is still its third power's, and what the
exponents hold."""
import pytest
import torch

from test_gpu_ortho import run, steps_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(3, 3), (3, 5), (7, 3), (100, 128), (200, 300), (300, 200)])
@pytest.mark.parametrize("c", [0.0, 1e-20, -1e-20, 1e-38])
def test_a_fifth_power_next_to_nothing(rows, cols, c):
    """Three singular values at 3^-0.5, where 2.6 s - 2.6 s^3 is largest, 1.0007.  To 2^-17: two steps of three products, each
    rounded to 2^-22 or less of terms that are at most three times the result."""
    g = torch.zeros(1, rows, cols)
    g[0, :3, :3] = torch.eye(3)
    coef = (2.6, -2.6, c, 1.5, -0.5, 0.0)
    got, ref = run(g, coef).double(), steps_of(g, coef, 1e-7, 1.0, torch.float64)
    assert float((got - ref).norm() / ref.norm()) <= 2.0 ** -17
