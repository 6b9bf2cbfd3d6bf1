"""Random draws over sizes, types, layouts and plans of the 4-bit product, its quantiser and the orthogonalised update, and
routings at the ends of what the losses take."""
import random

import pytest
import torch

import mx_util as U
import tensor_core_mixed_amd as T
import test_gpu_mxfp4 as G
import test_gpu_ortho as O
import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


def log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


@pytest.mark.parametrize("seed", range(80))
def test_products(seed):
    rng = random.Random(seed)
    M, N, K = log_size(rng, 1, 700), log_size(rng, 1, 700), log_size(rng, 1, 6000)
    c = rng.choice(G.TYPES)
    config, split = rng.choice([(-1, 0), (-1, 0), (rng.randint(0, 5), rng.choice([0, 1, 2, 5, 13]))])
    kw = dict(pad=(rng.randint(0, 2), rng.randint(0, 2), rng.randint(0, 5))) if rng.random() < 0.3 else {}
    with G.forced(fp4_config=config, fp4_split=split):
        G.check_gemm(M, N, K, c, *(rng.random() < 0.4 for _ in range(3)), spread=0 if c == torch.float16 else rng.choice([0, 3, 9]), seed=seed, **kw)


@pytest.mark.parametrize("seed", range(40))
def test_quantiser(seed):
    rng = random.Random(seed)
    x = G.normal(torch.Generator().manual_seed(seed), log_size(rng, 1, 700), log_size(rng, 1, 700), rng.choice(G.TYPES))
    G.check_quantize(x, rng.choice(["rows", "cols", "both"]), pad=rng.randint(0, 5), shift=rng.randint(0, 3))


@pytest.mark.parametrize("seed", range(40))
def test_updates(seed):
    rng = random.Random(seed)
    b, r, c = rng.choice([1, 1, 2, 5]), log_size(rng, 8, 700), log_size(rng, 8, 700)
    t = rng.choice(list(O.TYPES))
    g = O.update(torch.Generator().manual_seed(seed), b, r, c, t)
    O.check(g, coef=O.MUON * rng.randint(1, 5), scale=rng.choice([1.0, 0.2, 7.0]), out=rng.choice([t, torch.float32]), pad=rng.randint(0, 3),
            gap=rng.randint(0, 3), shift=rng.randint(0, 1))


@pytest.mark.parametrize("tokens", [5, 1000])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [0, 7, 300])
def test_no_slots(tokens, sigmoid, E):
    """Counts of nothing: no balance loss; without experts no z loss either."""
    x = torch.randn(tokens, E, generator=torch.Generator().manual_seed(1))
    mask = (torch.arange(tokens) % 5 != 0).to(torch.uint8)
    xb = x.cuda() if E else torch.zeros(tokens, 1, device="cuda")
    counts, losses = torch.full((E + 1,), -5, dtype=torch.int32, device="cuda"), torch.full((2,), 9.0, device="cuda")
    m = mask.cuda()
    assert T.tcm_moe_balance(tokens, E, 0, xb.data_ptr(), max(E, 1), T.TCM_F32_F32 | (T.TCM_ROUTE_SIGMOID if sigmoid else 0), None, m.data_ptr(),
                             counts.data_ptr(), losses.data_ptr(), R.stream()) == T.TCM_OK
    torch.cuda.synchronize()
    assert (counts[:-1] == 0).all() and int(counts[-1]) == int(mask.sum()) and float(losses[0]) == 0
    z = float(torch.logsumexp(x[mask != 0].double(), 1).square().mean()) if E else 0.0
    assert abs(float(losses[1]) - z) <= 1e-5 * z


@pytest.mark.parametrize("tokens", [100, 3000])
def test_losses_of_a_load_on_one_expert(tokens):
    """All choices on one expert: the losses' largest (experts), and, on an expert that the scores give e^-30, a small one, to 2^-34."""
    E, k = 1024, 1
    x = torch.zeros(tokens, E)
    x[:, 3] = 60.0
    for chosen, share in ((3, 1.0), (5, float(torch.exp(torch.tensor(-60.0).double())))):
        ids = torch.full((tokens, k), chosen, dtype=torch.int32)
        counts, losses = R.run_balance(x, ids, None, False)
        assert int(counts[chosen]) == tokens and int(counts[:-1].sum()) == tokens
        # (a few steps of binary32 in the share, and the sum's own 2^-34)
        assert abs(float(losses[0]) - E * share) <= E * share * 2.0 ** -20 + 2.0 ** -34
