"""The router's losses and their gradient against the formulas in 64 bits, and the gradient against differences."""
import math

import pytest
import torch

import tensor_core_mixed_amd as T

pytestmark = pytest.mark.gpu
TYPES = {torch.float32: T.TCM_F32_F32, torch.float16: T.TCM_F16_F32, torch.bfloat16: T.TCM_BF16_F32}
OUT_FLAG = {torch.float32: 0, torch.float16: T.TCM_C_F16, torch.bfloat16: T.TCM_C_BF16}
STEP = 2.0 ** -23


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return t.data_ptr() if t is not None else None


def keep_of(mask, tokens):
    return torch.ones(tokens, dtype=torch.bool) if mask is None else mask != 0


def shares(x, sigmoid):
    """p of every token (zeros for a token of nothing but -inf), float64."""
    ls = torch.nn.functional.logsigmoid(x) if sigmoid else x
    return torch.where((x == -math.inf).all(1, keepdim=True), 0.0, torch.softmax(ls, 1))


def loss_ref(x, ids, mask, sigmoid):
    """(counts, losses, their bounds).

    The bound: a share p is an exponential (its argument off by half a step of its size and of the largest logit's,
    its value by two steps), over a sum of up to 22 more roundings and a division; its mean has up to 80 additions
    (tokens of a wave, waves).  All are positive: relative errors add.  The log of a sum is off by a step of itself
    and of the largest logit, and the sum's relative error."""
    x = x.double()
    T_, E = x.shape
    keep = keep_of(mask, T_)
    live = keep & ~(x == -math.inf).all(1)
    good = ids[keep].long().flatten()
    good = good[(good >= 0) & (good < E)]
    counts = torch.bincount(good, minlength=E)
    n, k = max(1, int(keep.sum())), max(1, ids.shape[1])
    p = shares(x, sigmoid)
    loss = E * (counts.double() / (n * k) * p[keep].sum(0) / n).sum()
    lse = torch.logsumexp(x, 1)[live]
    z = lse.square().sum() / n
    finite = x[live][x[live] > -math.inf]
    reach = float(finite.max() - finite.min()) + float(finite.abs().max()) if len(finite) else 0.0
    dl = (reach + 110) * STEP * loss
    dz = (2 * lse.abs() * ((lse.abs() + reach + 30) * STEP)).sum() / n + 4 * STEP * z
    return torch.cat((counts, keep.sum()[None])).to(torch.int32), torch.stack((loss, z)), torch.stack((dl, dz)) + 1e-40


def run_balance(x, ids, mask, sigmoid, pad=0):
    tokens, E = x.shape
    xb = torch.full((tokens, E + pad), 50.0, dtype=x.dtype, device="cuda")
    xb[:, :E] = x.cuda()
    i, m = ids.cuda().contiguous(), mask.cuda() if mask is not None else None
    counts = torch.full((E + 2,), -5, dtype=torch.int32, device="cuda")
    losses = torch.full((3,), 9.0, device="cuda")
    st = T.tcm_moe_balance(tokens, E, ids.shape[1], xb.data_ptr(), E + pad, TYPES[x.dtype] | (T.TCM_ROUTE_SIGMOID if sigmoid else 0),
                           i.data_ptr(), ptr(m), counts.data_ptr(), losses.data_ptr(), stream())
    assert st == T.TCM_OK
    torch.cuda.synchronize()
    assert counts[-1] == -5 and losses[-1] == 9
    return counts[:-1].cpu(), losses[:-1].cpu()


def inputs(tokens, E, k, t, seed=0, spread=2.0, masked=False):
    gen = torch.Generator().manual_seed(seed + 31 * tokens + E)
    x = (spread * torch.randn(tokens, E, generator=gen)).to(t)
    ids = torch.topk(x.float(), k, dim=1)[1].to(torch.int32)
    mask = (torch.rand(tokens, generator=gen) > 0.3).to(torch.uint8) if masked else None
    return x, ids, mask


def check_balance(x, ids, mask, sigmoid, **kw):
    counts, losses = run_balance(x, ids, mask, sigmoid, **kw)
    want, ref, bound = loss_ref(x, ids, mask, sigmoid)
    assert torch.equal(counts, want)
    assert ((losses.double() - ref).abs() <= bound).all(), (losses, ref, bound)


@pytest.mark.parametrize("tokens", [1, 5, 128, 129, 1000, 5003])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (64, 6), (65, 1), (256, 8), (300, 64), (1024, 4)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance(tokens, E, k, sigmoid):
    t = list(TYPES)[(tokens + E) % 3]
    x, ids, mask = inputs(tokens, E, k, t, masked=tokens % 2 == 1)
    check_balance(x, ids, mask, sigmoid, pad=tokens % 3)


def far_inputs(tokens, E, k):
    """Rows with masked experts, nothing but -inf, far negative logits, and repeated or foreign ids."""
    x, ids, _ = inputs(tokens, E, k, torch.float32, seed=9)
    x[0::7, 1::2] = -math.inf
    x[1::7] = -math.inf
    x[2::7] -= 1000
    x[3::7] += 80
    ids[4::7, 1] = ids[4::7, 0]
    ids[5::7, 0], ids[6::7, 1] = -1, E
    return x, ids


@pytest.mark.parametrize("tokens", [14, 700])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_far_rows(tokens, sigmoid):
    x, ids = far_inputs(tokens, 12, 3)
    check_balance(x, ids, None, sigmoid)


@pytest.mark.parametrize("tokens", [40, 400])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_tokens_may_hold_anything(tokens, sigmoid):
    x, ids, mask = inputs(tokens, 70, 3, torch.float32, masked=True)
    x[mask == 0] = math.nan
    ids[mask == 0] = 1 << 30
    check_balance(x, ids, mask, sigmoid)
    check_grad(x, ids, mask, sigmoid, norm=True)
    mask[:] = 0
    counts, losses = run_balance(x, ids, mask, sigmoid)
    assert not counts.any() and not losses.any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("tokens", [3, 300])
def test_nan_and_infinite_logits(bad, tokens):
    x, ids, _ = inputs(tokens, 20, 2, torch.float32)
    x[1, 3] = bad
    counts, losses = run_balance(x, ids, None, False)
    assert torch.equal(counts, loss_ref(x, ids, None, False)[0]) and losses.isnan().all()
    d = run_grad(x, ids, None, False, True, torch.randn(tokens, 2), counts, torch.ones(2), 1.0, torch.float32)
    assert d[1].isnan().all() and not d[0].isnan().any() and not d[2:].isnan().any()


def test_no_tokens():
    ids = torch.zeros(0, 2, dtype=torch.int32)
    counts, losses = run_balance(torch.zeros(0, 5), ids, None, False)
    assert not counts.any() and not losses.any()


def grad_ref(x, ids, mask, sigmoid, norm, dw, counts, dl, scale):
    """(D, bound) in float64: the formulas, term by term.

    The bound: every term is a product of shares, whose relative error is that of an exponential and a sum (`reach`
    and 40 steps), times a difference of numbers weighted with shares, whose errors are relative to its parts' differences."""
    x = x.double()
    T_, E = x.shape
    keep = keep_of(mask, T_) & ~(x == -math.inf).all(1)
    x = torch.where(keep[:, None], x, 0.0)
    p, soft = shares(x, sigmoid), torch.softmax(x, 1)
    s, r = torch.sigmoid(x), torch.sigmoid(-x)
    finite = x[x > -math.inf]
    c = (float(finite.max() - finite.min()) + float(finite.abs().max()) + 40) * STEP
    d, m = torch.zeros_like(x), torch.zeros_like(x)

    def centred(w, v):
        """w_e (v_e - sum w v) and sum_i w_e w_i |v_e - v_i|, rows apart"""
        return w * (v - (w * v).sum(1, keepdim=True)), w * (w[:, None, :] * (v[:, :, None] - v[:, None, :]).abs()).sum(2)

    def add(value, size):
        nonlocal d, m
        d, m = d + value, m + size

    if dl is not None:
        n, k = max(1, int(counts[-1])), max(1, ids.shape[1])
        value, size = centred(p, counts[:-1].double().expand(T_, E) * (float(dl[0]) * E / (n * n * k)))
        f = r if sigmoid else 1.0
        add(f * value, f * size)
        z = float(dl[1]) * 2 / n * torch.logsumexp(x, 1, keepdim=True) * soft
        add(z, z.abs() + abs(float(dl[1])) * 2 / n * soft)
    if dw is not None:
        good = (ids >= 0) & (ids < E)
        at = torch.where(good, ids, 0).long()
        g = torch.where(good, dw.double(), 0.0)
        if norm:
            l = torch.where(good, (torch.nn.functional.logsigmoid(x) if sigmoid else x).gather(1, at), -math.inf)
            w = torch.where((l == -math.inf).all(1, keepdim=True), 0.0, torch.softmax(l, 1))
            value, size = centred(w, g)
            value, size = (torch.zeros_like(x).scatter_add(1, at, torch.where(good, scale * v, 0.0)) for v in (value, abs(scale) / scale * size))
            f = r if sigmoid else 1.0
            add(f * value, f * size.abs() * 1.0)
        else:
            G = torch.zeros_like(x).scatter_add(1, at, g)
            if sigmoid:
                add(scale * r * s * G, abs(scale) * r * s * torch.zeros_like(x).scatter_add(1, at, g.abs()))
            else:
                value, size = centred(p, G)
                add(scale * value, abs(scale) * size)
    d, m = (torch.where(keep[:, None], v, 0.0) for v in (d, m))
    return d, c * m + 1e-37


def run_grad(x, ids, mask, sigmoid, norm, dw, counts, dl, scale, d_type, pad=0):
    tokens, E = x.shape
    xb = torch.full((tokens, E + pad), 50.0, dtype=x.dtype, device="cuda")
    xb[:, :E] = x.cuda()
    D = torch.full((tokens, E + pad), 4.0, dtype=d_type, device="cuda")
    up = lambda v: v.cuda().contiguous() if v is not None else None
    i, m, w, n, l = up(ids), up(mask), up(dw), up(counts), up(dl)
    code = TYPES[x.dtype] | OUT_FLAG[d_type] | (T.TCM_ROUTE_SIGMOID if sigmoid else 0) | (T.TCM_ROUTE_NORM if norm else 0)
    st = T.tcm_moe_route_grad(tokens, E, ids.shape[1], xb.data_ptr(), E + pad, code, scale, ptr(i), ptr(m), ptr(w), ptr(n), ptr(l),
                              D.data_ptr(), E + pad, stream())
    assert st == T.TCM_OK
    torch.cuda.synchronize()
    assert (D[:, E:] == 4).all()
    return D[:, :E].cpu()


def check_grad(x, ids, mask, sigmoid, norm, weights=True, losses=True, scale=1.0, d_type=torch.float32, pad=0):
    tokens, k = ids.shape
    gen = torch.Generator().manual_seed(tokens)
    dw = torch.randn(tokens, k, generator=gen) if weights else None
    dl = torch.tensor([0.7 * tokens, -0.2 * tokens]) if losses else None
    counts = loss_ref(torch.nan_to_num(x.float()), ids, mask, sigmoid)[0] if losses else None
    got = run_grad(x, ids, mask, sigmoid, norm, dw, counts, dl, scale, d_type, pad)
    ref, bound = grad_ref(x, ids, mask, sigmoid, norm, dw, counts, dl, scale)
    f = torch.finfo(d_type)
    half = (ref.abs() + bound).clamp_min(f.smallest_normal) * f.eps / 2
    bad = (got.double() - ref).abs() > bound + half
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3], got[bad][:3], ref[bad][:3], bound[bad][:3])


@pytest.mark.parametrize("tokens", [1, 33, 500])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (64, 6), (65, 1), (256, 8), (300, 64), (1000, 4)])
@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, False), (True, True)])
def test_grad(tokens, E, k, sigmoid, norm):
    if tokens * E > 200000:
        tokens = 60  # (the reference takes every pair of experts)
    t = list(TYPES)[(tokens + E) % 3]
    x, ids, mask = inputs(tokens, E, k, t, masked=tokens % 2 == 1)
    check_grad(x, ids, mask, sigmoid, norm, scale=1.0 + k, pad=k % 3)


@pytest.mark.parametrize("d_type", list(TYPES))
@pytest.mark.parametrize("weights,losses", [(True, False), (False, True), (False, False)])
def test_grad_parts(d_type, weights, losses):
    x, ids, mask = inputs(50, 30, 4, d_type, masked=True)
    check_grad(x, ids, mask, True, True, weights, losses, scale=2.5, d_type=d_type)
    check_grad(x, ids, mask, False, False, weights, losses, scale=2.5, d_type=d_type)


@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, False), (True, True)])
def test_grad_far_rows(sigmoid, norm):
    x, ids = far_inputs(70, 12, 3)
    check_grad(x, ids, None, sigmoid, norm)


@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, True)])
def test_grad_where_one_expert_takes_all(sigmoid, norm):
    """p within 1e-6 of 1: what is left of differences counts."""
    x, ids, _ = inputs(40, 16, 2, torch.float32)
    x[torch.arange(40), ids[:, 0].long()] += 14
    check_grad(x, ids, None, sigmoid, norm)


@pytest.mark.parametrize("sigmoid,norm", [(False, False), (False, True), (True, False), (True, True)])
def test_grad_against_differences(sigmoid, norm):
    """The losses and weights themselves in 64 bits, moved along a direction."""
    tokens, E, k, scale = 20, 11, 3, 1.5
    x, ids, mask = inputs(tokens, E, k, torch.float32, masked=True)
    gen = torch.Generator().manual_seed(4)
    dw, dl = torch.randn(tokens, k, generator=gen), torch.tensor([30.0, -5.0])
    counts, _ = run_balance(x, ids, mask, sigmoid)
    keep = keep_of(mask, tokens)

    def total(x):
        score = torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)
        w = score.gather(1, ids.long())
        w = scale * (w / w.sum(1, keepdim=True) if norm else w)
        loss = loss_ref(x, ids, mask, sigmoid)[1]
        return float((w * dw)[keep].sum() + (loss * dl.double()).sum())

    d = run_grad(x, ids, mask, sigmoid, norm, dw, counts, dl, scale, torch.float32).double()
    v = torch.randn(tokens, E, generator=gen).double()
    h = 1e-4
    want = (8 * (total(x.double() + h * v) - total(x.double() - h * v)) - (total(x.double() + 2 * h * v) - total(x.double() - 2 * h * v))) / (12 * h)
    # differences: a fifth derivative of order 10 at most times h^4 / 30, and 64-bit rounding over h; the gradient: its bound
    bound = float((grad_ref(x, ids, mask, sigmoid, norm, dw, counts, dl, scale)[1] * v.abs()).sum()) + 1e-9 * float(dw.abs().sum() + 100)
    assert abs(float((d * v).sum()) - want) <= bound


def test_the_same_call_gives_the_same_bits():
    x, ids, _ = inputs(6000, 256, 8, torch.bfloat16)
    first = run_balance(x, ids, None, True)
    for _ in range(3):
        again = run_balance(x, ids, None, True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_route_then_losses_then_gradient_in_a_graph():
    """The router's training step as one captured graph, replayed on other logits with eager work between."""
    tokens, E, k = 700, 64, 4
    x = torch.empty(tokens, E, device="cuda")
    ids, w = torch.empty(tokens, k, dtype=torch.int32, device="cuda"), torch.empty(tokens, k, device="cuda")
    counts, losses = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    dw, dl, D = torch.randn(tokens, k, device="cuda"), torch.ones(2, device="cuda"), torch.empty(tokens, E, device="cuda")

    def step(s):
        for st in (T.tcm_moe_route(tokens, E, k, x.data_ptr(), E, T.TCM_F32_F32 | T.TCM_ROUTE_NORM, None, 1.0, ids.data_ptr(), w.data_ptr(), s),
                   T.tcm_moe_balance(tokens, E, k, x.data_ptr(), E, T.TCM_F32_F32, ids.data_ptr(), None, counts.data_ptr(), losses.data_ptr(), s),
                   T.tcm_moe_route_grad(tokens, E, k, x.data_ptr(), E, T.TCM_F32_F32 | T.TCM_ROUTE_NORM, 1.0, ids.data_ptr(), None,
                                        dw.data_ptr(), counts.data_ptr(), dl.data_ptr(), D.data_ptr(), E, s)):
            assert st == T.TCM_OK

    side = torch.cuda.Stream()
    gen = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda: torch.randn(tokens, E, generator=gen, device="cuda")
    x.copy_(draw())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(side.cuda_stream)  # (the workspace grows)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(side.cuda_stream)
        for _ in range(4):
            x.copy_(draw())
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (ids, w, counts, losses, D)]
            step(side.cuda_stream)
            torch.cuda.synchronize()
            for a, b in zip(got, (ids, w, counts, losses, D)):
                assert torch.equal(a, b)
