"""The update of matrices whose parts differ in size: what one exponent a matrix leaves of the smaller part's bits."""
import pytest
import torch

from test_gpu_ortho import run, steps_of, update

pytestmark = pytest.mark.gpu
CUBIC = (1.5, -0.5, 0.0)  # (singular values go to 1, the small ones half as large again a step)


def two_parts(n, m, p, across):
    """A matrix of normal values over one of them times 2^-p, in columns of their own; the second's rows and columns."""
    g = torch.zeros(1, 2 * n, 2 * m)
    a, b = torch.randn(2, n, m, generator=torch.Generator().manual_seed(p))
    g[0, :n, :m], g[0, n:, m:] = a, b * 2.0 ** -p
    return g.mT.contiguous() if across else g


@pytest.mark.parametrize("n,m", [(32, 48), (100, 150)])
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("p,steps", [(4, 10), (12, 25), (16, 33), (20, 40), (20, 5)])
def test_a_part_below_the_norm(n, m, across, p, steps):
    """The bound on X stays 1.001 (2^13 in the parts), so a step rounds its values to 2^-38 at least.  The parts share neither
    rows nor columns: such errors of the small one grow like itself, at most by 1 / s, s its least singular value at the time,
    which grows by 1.5 a step: 3 sqrt(n m) 2^-38 / s in all, s the first one.  Besides, the bound of test_gpu_ortho.check."""
    g = two_parts(n, m, p, across)
    got, ref = run(g, CUBIC * steps)[0].double(), steps_of(g, CUBIC * steps, 1e-7, 1.0, torch.float64)[0]
    single = steps_of(g, CUBIC * steps, 1e-7, 1.0, torch.float32)[0].double()
    if across:
        g, got, ref, single = g.mT, got.T, ref.T, single.T
    x = g[0].double() / g[0].double().norm()
    least = float(torch.linalg.svdvals(x[n:, m:]).min())
    for at, floor in (((slice(0, n), slice(0, m)), 0.0), ((slice(n, None), slice(m, None)), 3 * (n * m) ** 0.5 * 2.0 ** -38 / least)):
        off = float((got[at] - ref[at]).norm())
        bound = 4 * float((single[at] - ref[at]).norm()) + 2.0 ** -20 * float(ref[at].norm()) + min(floor, 1.5 ** steps * 3 * (n * m) ** 0.5 * 2.0 ** -38)
        assert off <= bound, (off, bound)
    assert not got[:n, m:].any() and not got[n:, :m].any()


@pytest.mark.parametrize("n,m", [(32, 48), (100, 150)])
def test_a_part_below_the_range(n, m):
    """Values under 2^-39 of the norm count as zeros."""
    g = two_parts(n, m, 46, False)
    got = run(g, CUBIC * 80)[0]
    assert not got[n:].any()
    s = torch.linalg.svdvals(got[:n, :m].double())
    assert float((s - 1).abs().max()) < 2.0 ** -18  # (roundings of 2^-22 a step, which each step halves or better)


@pytest.mark.parametrize("shape", [(1, 64, 96), (1, 200, 300)])
@pytest.mark.parametrize("factor", [2.0 ** -8, 2.0 ** -16])
def test_an_eps_above_the_norm(shape, factor):
    """X starts at `factor` of its bound: values are rounded to 2^-38 of it where they are that small.  One step takes
    singular values by 3.5 at most, five by less than 600."""
    g = update(torch.Generator().manual_seed(1), *shape, torch.float32, 1.0)
    eps = float(torch.tensor(float(g.double().norm()) / factor))
    coef = (3.4445, -4.7750, 2.0315) * 5
    got, ref = run(g, coef, eps)[0].double(), steps_of(g, coef, eps, 1.0, torch.float64)[0]
    single = steps_of(g, coef, eps, 1.0, torch.float32)[0].double()
    n, m = shape[1:]
    # (2^-36: the bound on X lies between 1 and 2 after a step; an error grows by the rest of 3.4445^5 = 485)
    floor = sum(3.4445 ** k for k in range(6)) * (n * m) ** 0.5 * 2.0 ** -36
    off = float((got - ref).norm())
    assert off <= 4 * float((single - ref).norm()) + 2.0 ** -20 * float(ref.norm()) + floor
