"""The orthogonalised update of matrices with a shorter side of at most 128 (a workgroup's chunk of columns holds them):
chunks' edges, both ways round, many steps, entries by the hundred, sides next to the limits."""
import pytest
import torch

import tensor_core_mixed_amd as T
from test_gpu_ortho import MUON, check, run, steps_of, update

pytestmark = pytest.mark.gpu
SMALL = [(1, 256), (17, 257), (32, 255), (33, 512), (63, 900), (64, 256), (64, 8192), (65, 65), (65, 128), (96, 129), (127, 384), (128, 128), (128, 1024)]
LARGE = [(64, 8193), (65, 1025), (128, 1025), (129, 129), (129, 300)]


@pytest.mark.parametrize("n,m", SMALL + LARGE)
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("t,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
def test_chunks(n, m, tall, t, out):
    g = update(torch.Generator().manual_seed(n * 10007 + m), 2, *((m, n) if tall else (n, m)), t)
    check(g, out=out, pad=3, gap=5, shift=1)
    assert ("kernel=ortho_small" in T.tcm_last_plan()) == ((n, m) in SMALL)


@pytest.mark.parametrize("shape", [(2, 40, 100), (2, 300, 50), (1, 100, 300)])
@pytest.mark.parametrize("steps", [1, 2, 16, 17, 33])
def test_steps(shape, steps):
    """(1.5, -0.5, 0) leads to the nearest orthogonal matrix; a well-conditioned one, so that all steps matter and none ends at 0."""
    gen = torch.Generator().manual_seed(steps)
    b, r, c = shape
    g = torch.randn(shape, generator=gen) + 3 * torch.eye(r, c)[None]
    check(g, coef=(1.5, -0.5, 0.0) * steps, scale=0.3)
    check(g, coef=MUON * min(steps, 6), scale=-2.0)


@pytest.mark.parametrize("shape", [(700, 20, 30), (300, 90, 60), (40, 500, 64), (33, 128, 600)])
def test_many_entries(shape):
    check(update(torch.Generator().manual_seed(3), *shape, torch.bfloat16))


@pytest.mark.parametrize("shape", [(3, 50, 60), (3, 50, 700), (3, 700, 100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_stays_in_its_entry(shape, bad):
    g = update(torch.Generator().manual_seed(4), *shape, torch.float32)
    clean = run(g)
    g[1, 30, 40] = bad
    got = run(g)
    assert got[1].isnan().all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


@pytest.mark.parametrize("shape", [(3, 50, 60), (3, 50, 700), (3, 700, 100)])
def test_sizes_of_values(shape):
    """An entry of zeros gives zeros; a factor far from 1, up to binary32's ends, changes nothing but rounding."""
    g = update(torch.Generator().manual_seed(5), *shape, torch.float32, 1.0)
    g[1] = 0
    check(g)
    assert (run(g)[1] == 0).all()
    base = run(g, eps=0.0)
    for f in (2.0 ** -100, 2.0 ** 100):
        assert torch.equal(run(f * g, eps=0.0)[0], base[0]) and torch.equal(run(f * g, eps=0.0)[2], base[2])


@pytest.mark.parametrize("shape", [(2, 30, 40), (2, 150, 200)])
@pytest.mark.parametrize("coef", [(2.0 ** 38, 0.0, 0.0, 2.0 ** -38, 0.0, 0.0), (2.0 ** -38, 0.0, 0.0, 2.0 ** 38, 0.0, 0.0), (0.0, 2.0 ** -70, 0.0),
                                  (1.0, 2.0 ** 60, 0.0), (0.0, 0.0, 2.0 ** -75), (0.0, 0.0, 0.0, 1.0, 1.0, 1.0)])
def test_coefficients_far_from_1(shape, coef):
    """To 2^-20 (roundings of 2^-22, none of them amplified in one or two steps), also where the same steps in binary32
    would leave its range (the fourth power of 2^38)."""
    g = torch.randn(shape, generator=torch.Generator().manual_seed(6))
    got, ref = run(g, coef).double(), steps_of(g, coef, 1e-7, 1.0, torch.float64)
    assert ((got - ref).square().sum((1, 2)).sqrt() <= 2.0 ** -20 * ref.square().sum((1, 2)).sqrt()).all()
