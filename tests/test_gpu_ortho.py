"""The orthogonalised update against its steps in 64 bits."""
import pytest
import torch

import tensor_core_mixed_amd as T

pytestmark = pytest.mark.gpu
TYPES = {torch.float32: T.TCM_F32_F32, torch.float16: T.TCM_F16_F32, torch.bfloat16: T.TCM_BF16_F32}
OUT_FLAG = {torch.float32: 0, torch.float16: T.TCM_C_F16, torch.bfloat16: T.TCM_C_BF16}
MUON = (3.4445, -4.7750, 2.0315)


def steps_of(G, coef, eps, scale, dtype):
    """The formula in `dtype` on the CPU, (batch, rows, cols)."""
    x = G.double()
    x = (x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)).to(dtype)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    for a, b, c in zip(coef[0::3], coef[1::3], coef[2::3]):
        a, b, c = (float(torch.tensor(v)) for v in (a, b, c))  # (as binary32 holds them)
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return scale * (x.mT if tall else x)


def run(G, coef=MUON * 5, eps=1e-7, scale=1.0, out=torch.float32, pad=0, gap=0, shift=0):
    """O of a call whose matrices lie in wider rows, apart by more, from an address `shift` elements past an aligned one."""
    b, r, c = G.shape
    ld, st = c + pad, r * (c + pad) + gap
    gbuf = torch.full((b * st + shift,), 3.0, dtype=G.dtype)
    for e in range(b):
        gbuf[shift + e * st:shift + e * st + r * ld].view(r, ld)[:, :c] = G[e]
    obuf = torch.full((b * st + shift,), 5.0, dtype=out, device="cuda")
    g = gbuf.cuda()
    st_ = T.tcm_orthogonalize(b, r, c, g[shift:].data_ptr(), ld, st, obuf[shift:].data_ptr(), ld, st, TYPES[G.dtype] | OUT_FLAG[out], coef, eps,
                              scale, torch.cuda.current_stream().cuda_stream)
    assert st_ == T.TCM_OK
    torch.cuda.synchronize()
    o = obuf.cpu()
    got = torch.stack([o[shift + e * st:shift + e * st + r * ld].view(r, ld)[:, :c] for e in range(b)])
    kept = torch.ones(b * st + shift, dtype=torch.bool)
    for e in range(b):
        kept[shift + e * st:shift + e * st + r * ld].view(r, ld)[:, :c] = False
    assert (o[kept] == 5).all()
    return got


def check(G, coef=MUON * 5, eps=1e-7, scale=1.0, out=torch.float32, **kw):
    """Entry by entry, by the norm of the difference.

    The bound: a value in two parts is off by 2^-23 of itself, binary32's by 2^-25, a product without lower times lower by
    2^-22 of its terms' sizes, binary32's by 2^-24 a term; every rounding is at most four times that of the same steps in
    binary32, so the error is held to four times theirs (their own error is what a CPU makes of them), and as that may be
    small by chance, to 2^-20 of the result besides; for sizes under 8, where a few roundings stand alone, to 2^-16: three
    roundings of 2^-22 a step, up to 9 times larger where a x and the rest nearly cancel, five steps.  Then O's own rounding."""
    got = run(G, coef, eps, scale, out, **kw).double()
    ref = steps_of(G, coef, eps, scale, torch.float64)
    single = steps_of(G, coef, eps, scale, torch.float32).double()
    norm = lambda x: x.square().sum((1, 2)).sqrt()
    least = 2.0 ** (-16 if min(G.shape[1:]) < 8 else -20)
    f = torch.finfo(out)
    half = f.eps / 2 * norm(ref) + f.smallest_normal * f.eps * (G.shape[1] * G.shape[2]) ** 0.5
    bound = 4 * norm(single - ref) + least * norm(ref) + half
    off = norm(got - ref)
    assert (off <= bound).all(), (off / norm(ref), bound / norm(ref), T.tcm_last_plan())


def update(gen, b, r, c, t, size=1e-3):
    """A few strong directions over noise."""
    g = torch.randn(b, r, c, generator=gen) + torch.randn(b, r, 3, generator=gen) @ torch.randn(b, 3, c, generator=gen)
    return (size * g).to(t)


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 5, 3), (1, 31, 33), (4, 64, 64), (2, 100, 257), (2, 257, 100), (1, 128, 512), (1, 130, 1000), (1, 1000, 96),
          (3, 600, 300), (1, 513, 514), (20, 40, 24), (1, 33, 3000)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", list(TYPES))
def test_against_64_bits(shape, t):
    gen = torch.Generator().manual_seed(sum(shape))
    G = update(gen, *shape, t)
    check(G)
    if t != torch.float32:
        check(G, out=t, scale=0.2 * max(shape[1:]) ** 0.5)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("pad,gap,shift", [(1, 3, 1), (8, 0, 0), (0, 5, 3)])
@pytest.mark.parametrize("shape", [(3, 70, 45), (3, 45, 70)])
def test_strides(shape, t, pad, gap, shift):
    G = update(torch.Generator().manual_seed(1), *shape, t)
    check(G, out=t, pad=pad, gap=gap, shift=shift)


def test_large_tiles():
    G = update(torch.Generator().manual_seed(2), 2, 1100, 2700, torch.bfloat16)
    check(G, out=torch.bfloat16)


@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e30, 1e36])
def test_far_sizes(size):
    check(update(torch.Generator().manual_seed(3), 2, 50, 80, torch.float32, size), eps=0.0)


@pytest.mark.parametrize("coef", [(1.5, -0.5, 0.0) * 6, (8.28, -23.6, 17.3, 4.1, -2.9, 0.55, 3.9, -2.8, 0.55, 1.9, -1.3, 0.4), (0.5, 0.0, 0.0) * 3,
                                  (0.0, 0.0, 1.0), (0.0, 1.0, 0.0, 2.0, 0.0, 0.0), (-300.0, 500.0, 1e4)])
def test_coefficients(coef):
    check(update(torch.Generator().manual_seed(4), 2, 60, 90, torch.float32), coef)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("shape", [(2, 3, 5), (2, 130, 70)])
def test_no_steps(shape, t):
    G = update(torch.Generator().manual_seed(5), *shape, t)
    got = run(G, (), 1e-3, 2.0, t, pad=1)
    ref = steps_of(G, (), 1e-3, 2.0, torch.float64)
    f = torch.finfo(t)
    # (eps itself is held in binary32: 2^-24 of what is divided by)
    assert ((got.double() - ref).abs() <= ref.abs().clamp_min(f.smallest_normal) * f.eps / 2 * 1.01 + ref.abs() * 2.0 ** -22).all()


def test_zeros_and_equal_rows():
    G = update(torch.Generator().manual_seed(6), 3, 40, 60, torch.float32)
    G[0] = 0
    G[1, 20:] = G[1, :20]
    check(G)
    assert not run(G)[0].any()
    assert run(G, eps=0.0)[0].isnan().all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(3, 40, 70), (3, 70, 40)])
def test_nan_stays_in_its_entry(bad, shape):
    G = update(torch.Generator().manual_seed(7), *shape, torch.float32)
    G[1, 7, 9] = bad
    got = run(G)
    assert got[1].isnan().all()
    assert torch.equal(got[[0, 2]], run(G[[0, 2]]))


def test_the_same_bits_again_and_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(8)
    b, r, c = 2, 200, 700
    g, o = torch.empty(b, r, c, device="cuda"), torch.empty(b, r, c, device="cuda")

    def step(s):
        assert T.tcm_orthogonalize(b, r, c, g.data_ptr(), c, r * c, o.data_ptr(), c, r * c, T.TCM_F32_F32, MUON * 5, 1e-7, 1.0, s) == T.TCM_OK

    side = torch.cuda.Stream()
    g.copy_(torch.randn(b, r, c, generator=gen, device="cuda"))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(side.cuda_stream)  # (the workspace grows)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(side.cuda_stream)
        for _ in range(4):
            g.copy_(torch.randn(b, r, c, generator=gen, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            got = o.clone()
            step(side.cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(got, o)


def test_singular_values_end_near_one():
    """What the steps are for."""
    G = update(torch.Generator().manual_seed(9), 1, 100, 300, torch.float32)
    s = torch.linalg.svdvals(run(G, MUON * 7)[0].double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3
