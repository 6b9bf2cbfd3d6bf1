"""The expert router and the mixture-of-experts layer on the GPU against 64-bit references."""
import math

import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, X_CODE, blocks, check_close, half_step, moe_ref, quantize

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ router

def run_route(x, k, sigmoid=False, norm=False, bias=None, scale=1.0, ldx=None, shift=0):
    tok, E = x.shape
    ldx = ldx or E
    es = x.element_size()
    xv = torch.full((tok, ldx), float("nan"), dtype=x.dtype)
    xv[:, :E] = x
    buf = torch.cat([torch.zeros(shift, dtype=torch.uint8), xv.view(torch.uint8).flatten(), torch.zeros(8, dtype=torch.uint8)]).cuda()
    ids = torch.full((tok + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((tok + 1, k), -7.0, device="cuda")
    b = bias.float().cuda() if bias is not None else None
    code = X_CODE[x.dtype] | (T.TCM_ROUTE_SIGMOID if sigmoid else 0) | (T.TCM_ROUTE_NORM if norm else 0)
    st = T.tcm_moe_route(tok, E, k, buf.data_ptr() + shift, ldx, code, b.data_ptr() if b is not None else None, scale, ids.data_ptr(),
                         w.data_ptr(), stream())
    assert st == T.TCM_OK, T.tcm_status_string(st)
    torch.cuda.synchronize()
    assert (ids[tok] == -7).all() and (w[tok] == -7).all()
    return ids[:tok].cpu(), w[:tok].cpu()


def ref_route(x, k, sigmoid=False, norm=False, bias=None, scale=1.0):
    x = x.double()
    score = torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)
    key = x if bias is None else score + bias.double()
    ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
    w = score.gather(1, ids)
    return ids.to(torch.int32), (w / w.sum(1, keepdim=True) if norm else w) * scale


def check_route(x, k, **kw):
    ids, w = run_route(x, k, **kw)
    kw.pop("ldx", None), kw.pop("shift", None)
    rid, rw = ref_route(x, k, **kw)
    assert torch.equal(ids, rid)
    # exponents of arguments up to the row's range, a sum over the experts and one over the chosen ones, in binary32
    span = float(x.double().max() - x.double().min()) + float(x.double().abs().max()) + 1
    rel = 2 * (span + 16 + x.shape[1] / 64 + k) * 2.0 ** -24
    check_close(w, rw, rw.abs() * rel + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 4), (8, 2), (37, 5), (64, 6), (65, 10), (128, 8), (200, 7), (256, 8), (384, 10), (700, 64), (1024, 33)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route(dtype, E, k, sigmoid):
    gen = torch.Generator().manual_seed(E)
    x = (2 * torch.randn(70, E, generator=gen)).to(dtype)
    b = 0.1 * torch.randn(E, generator=gen)
    for norm in (False, True):
        check_route(x, k, sigmoid=sigmoid, norm=norm)
        check_route(x, k, sigmoid=sigmoid, norm=norm, bias=b, scale=2.5)


def test_route_many_tokens():
    x = torch.randn(5003, 60, generator=torch.Generator().manual_seed(1))
    check_route(x, 4, norm=True)


@pytest.mark.parametrize("E", [16, 64, 256, 300])
def test_route_ties_go_to_the_lower_expert(E):
    gen = torch.Generator().manual_seed(2)
    x = torch.randint(-2, 3, (64, E), generator=gen).float()
    x[0] = 0
    x[1] = -0.0
    x[1, ::2] = 0.0
    check_route(x, 8)
    check_route(x, 8, sigmoid=True, bias=torch.zeros(E))
    check_route(x.to(torch.bfloat16), 8, bias=torch.randint(0, 2, (E,), generator=gen).float(), norm=True)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_near_keys(sigmoid):
    """Keys that binary32 cannot tell apart: score + bias differ by less than its step."""
    gen = torch.Generator().manual_seed(3)
    E = 256
    x = torch.randn(512, E, generator=gen) * 0.5
    s = (torch.sigmoid(x.double()) if sigmoid else torch.softmax(x.double(), 1))[0]
    bias = (1.0 - s).float()  # row 0: every key within half a binary32 step of 1
    check_route(x, 10, sigmoid=sigmoid, bias=bias, norm=True)
    check_route(x[:1].expand(200, E).contiguous(), 10, sigmoid=sigmoid, bias=bias)


def test_route_far_logits():
    x = torch.tensor([[1e4, -1e4, 0.0, 9999.0], [-3e38, 3e38, 1.0, 2.0], [-100.0, -101.0, -102.0, -103.0]])
    for sigmoid in (False, True):
        ids, w = run_route(x, 4, sigmoid=sigmoid)
        rid, rw = ref_route(x, 4, sigmoid=sigmoid)
        assert torch.equal(ids, rid)
        # a score's argument carries half a step of its own size where the logits are far apart
        check_close(w, rw, rw * 2.0 ** -14 + 2.0 ** -126)


@pytest.mark.parametrize("E", [8, 100])
def test_route_masked_experts(E):
    """-inf logits: never chosen before a finite one, weight zero; a row of them alone gives weights of zero."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(6, E, generator=gen)
    x[0, 3:] = float("-inf")
    x[1] = float("-inf")
    x[2, :-1] = torch.finfo(torch.float32).min
    for sigmoid in (False, True):
        for norm in (False, True):
            ids, w = run_route(x, 5, sigmoid=sigmoid, norm=norm)
            assert torch.equal(ids[0, :3].sort()[0], torch.tensor([0, 1, 2], dtype=torch.int32)) and torch.equal(ids[0, 3:], torch.tensor([3, 4], dtype=torch.int32))
            assert (w[0, 3:] == 0).all() and (w[0, :3] > 0).all()
            assert torch.equal(ids[1], torch.arange(5, dtype=torch.int32)) and (w[1] == 0).all()
            rid, rw = ref_route(x[2:], 5, sigmoid=sigmoid, norm=norm)
            assert torch.equal(ids[2:], rid)
            check_close(w[2:], rw, rw * 2.0 ** -17 + 2.0 ** -126)


def test_route_nan_ranks_first():
    x = torch.randn(3, 70, generator=torch.Generator().manual_seed(5))
    x[1, 66] = float("nan")
    ids, w = run_route(x, 3, sigmoid=True)
    assert ids[1, 0] == 66 and w[1, 0].isnan() and not w[1, 1:].isnan().any()
    rid, rw = ref_route(x[[0, 2]], 3, sigmoid=True)
    assert torch.equal(ids[[0, 2]], rid)
    ids, w = run_route(x, 3)
    assert ids[1, 0] == 66 and w[1].isnan().all() and not w[[0, 2]].isnan().any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_any_alignment(dtype):
    x = torch.randn(9, 77, generator=torch.Generator().manual_seed(6)).to(dtype)
    for ldx, shift in ((77, 1), (80, 2), (91, 3)):
        check_route(x, 6, ldx=ldx, shift=shift)


# ------------------------------------------------------------------ expert layer

def make_moe(tok, H, I, E, k, dtype, w8, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = (spread * torch.randn(tok, H, generator=gen)).to(dtype)
    w1, w2 = torch.randn(E, 2, I, H, generator=gen) * H ** -0.5, torch.randn(E, H, I, generator=gen) * max(I, 1) ** -0.5
    s1 = s2 = None
    if w8:
        a = [[quantize(w1[e, i], E4M3, True) for i in range(2)] for e in range(E)]
        b = [quantize(w2[e], E4M3, True) for e in range(E)]
        w1, s1 = torch.stack([torch.stack([v[0] for v in r]) for r in a]).to(E4M3), torch.stack([torch.stack([v[1] for v in r]) for r in a])
        w2, s2 = torch.stack([v[0] for v in b]).to(E4M3), torch.stack([v[1] for v in b])
    else:
        w1, w2 = w1.to(dtype), w2.to(dtype)
    score = torch.rand(tok, E, generator=gen)
    wt, ids = torch.topk(score, k, dim=1)
    return x, ids.to(torch.int32), wt / wt.sum(1, keepdim=True), w1, s1, w2, s2


def run_moe(x, ids, wt, w1, s1, w2, s2, ldx=None, ldo=None, shift=0):
    tok, H = x.shape
    E, I = w1.shape[0], w1.shape[2]
    ldx, ldo = ldx or H, ldo or H
    sh = lambda t: torch.cat([torch.zeros(shift, dtype=torch.uint8), t.contiguous().view(torch.uint8).flatten()]).cuda()
    xp = torch.full((tok, ldx), float("nan"), dtype=x.dtype)
    xp[:, :H] = x
    xd, w1d, w2d = sh(xp), sh(w1), sh(w2)
    out = sh(torch.full((tok + 1, ldo), 3.0, dtype=x.dtype))
    dev = lambda t: t.contiguous().cuda() if t is not None else None
    idd, wd, s1d, s2d = dev(ids), dev(wt.float()), dev(s1), dev(s2)
    code = (T.TCM_F16_F32 | T.TCM_C_F16) if x.dtype == torch.float16 else (T.TCM_BF16_F32 | T.TCM_C_BF16)
    ptr = lambda t: t.data_ptr() if t is not None else None
    st = T.tcm_moe(tok, H, I, E, ids.shape[1], xd.data_ptr() + shift, ldx, idd.data_ptr(), wd.data_ptr(), w1d.data_ptr() + shift,
                   ptr(s1d), w2d.data_ptr() + shift, ptr(s2d), out.data_ptr() + shift, ldo,
                   code | (T.TCM_W_E4M3 if s1 is not None else 0), stream())
    assert st == T.TCM_OK, T.tcm_status_string(st)
    torch.cuda.synchronize()
    o = out.cpu()[shift:].view(x.dtype).view(tok + 1, ldo)
    assert (o[tok] == 3).all() and (o[:, H:] == 3).all(), "written past the output"
    return o[:tok, :H]


def check_moe(args, **kw):
    got = run_moe(*args, **kw)
    ref, bound = moe_ref(*args)
    check_close(got, ref, bound + half_step(ref, got.dtype) * (1 + 2.0 ** -10) + 2.0 ** -126)


SIZES = [(1, 64, 32, 4, 1), (1, 512, 256, 8, 8), (3, 264, 40, 5, 2), (7, 520, 136, 16, 3), (16, 128, 128, 4, 4), (17, 384, 264, 4, 2),
         (40, 256, 64, 3, 2), (64, 512, 96, 2, 1), (70, 136, 72, 6, 3), (5, 1000, 200, 40, 6)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("w8", [False, True])
def test_moe(size, dtype, w8):
    check_moe(make_moe(*size, dtype, w8, seed=size[0]))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("w8", [False, True])
def test_moe_odd_sizes_and_alignment(dtype, w8):
    for size in ((2, 77, 33, 4, 2), (5, 131, 130, 3, 3)):
        check_moe(make_moe(*size, dtype, w8))
    args = make_moe(4, 256, 64, 4, 2, dtype, w8)
    for kw in (dict(ldx=264, ldo=260), dict(ldx=259), dict(shift=2), dict(shift=8), dict(ldo=257)):
        check_moe(args, **kw)


@pytest.mark.parametrize("w8", [False, True])
def test_moe_all_tokens_on_one_expert(w8):
    args = list(make_moe(50, 256, 128, 8, 2, torch.bfloat16, w8))
    args[1][:] = torch.tensor([5, 2], dtype=torch.int32)
    check_moe(args)
    args[1][:] = 3  # an expert twice in a token's choice
    check_moe(args)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_moe_ids_out_of_range_add_nothing(dtype):
    args = list(make_moe(6, 256, 128, 8, 3, dtype, False))
    args[1][0] = torch.tensor([-1, 8, 1 << 30], dtype=torch.int32)  # a token without experts
    args[1][1, 1] = -5
    args[1][4, 0] = 100
    check_moe(args)
    assert (run_moe(*args)[0] == 0).all()
    args[1][:] = -1
    assert (run_moe(*args) == 0).all()


def test_moe_without_slots_or_inter():
    for size in ((3, 64, 32, 4, 0), (3, 64, 0, 4, 2)):
        assert (run_moe(*make_moe(*size, torch.bfloat16, False)) == 0).all()


def test_moe_zero_and_negative_weights():
    args = list(make_moe(5, 128, 64, 6, 3, torch.float16, False))
    args[2] = args[2] * torch.tensor([-1.0, 0.0, 2.0])
    check_moe(args)


@pytest.mark.parametrize("w8", [False, True])
def test_moe_products_past_the_16_bit_range(w8):
    """silu(g) u up to 10^8 between the two matrices of an f16 layer whose outputs are ordinary."""
    args = list(make_moe(6, 256, 96, 4, 2, torch.float16, w8, spread=100.0))
    if w8:
        args[4] = args[4] * 100
        args[6] = args[6] * 2.0 ** -20
    else:
        args[3] = (args[3].float() * 100).to(torch.float16)
        args[2] = args[2] * 2.0 ** -14
        args[5] = (args[5].float() * 2.0 ** -6).to(torch.float16)
    ref, _ = moe_ref(*args)
    assert ref.abs().max() < 60000
    check_moe(args)


def test_moe_nan_stays_in_its_token():
    args = list(make_moe(9, 256, 128, 4, 2, torch.bfloat16, False))
    args[0][4, 100] = float("nan")
    got = run_moe(*args)
    assert got[4].isnan().all()
    keep = [t for t in range(9) if t != 4]
    ref, bound = moe_ref(*[a[keep] if i < 3 else a for i, a in enumerate(args)])
    check_close(got[keep], ref, bound + half_step(ref, got.dtype) * (1 + 2.0 ** -10) + 2.0 ** -126)


@pytest.mark.parametrize("w8", [False, True])
def test_moe_repeats_and_graph(w8):
    """The same bits from call to call and from a captured graph, whose inputs change between replays."""
    x, ids, wt, w1, s1, w2, s2 = make_moe(12, 512, 256, 8, 4, torch.bfloat16, w8)
    d = lambda t: t.contiguous().cuda() if t is not None else None
    X, I, W, W1, S1, W2, S2 = map(d, (x, ids, wt.float(), w1, s1, w2, s2))
    out = torch.empty_like(X)
    ptr = lambda t: t.data_ptr() if t is not None else None
    code = T.TCM_BF16_F32 | T.TCM_C_BF16 | (T.TCM_W_E4M3 if w8 else 0)

    def call():
        assert T.tcm_moe(12, 512, 256, 8, 4, X.data_ptr(), 512, I.data_ptr(), W.data_ptr(), W1.data_ptr(), ptr(S1), W2.data_ptr(),
                         ptr(S2), out.data_ptr(), 512, code, stream()) == T.TCM_OK
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        for i in range(4):
            I.copy_((I + i) % 8)
            out.zero_()
            call()
            eager = out.clone()
            out.zero_()
            g.replay()
            s.synchronize()
            assert torch.equal(out, eager)


def test_route_feeds_the_layer():
    """Logits through the router into the layer, as a model calls them, against the same in 64 bits."""
    x, _, _, w1, s1, w2, s2 = make_moe(10, 256, 128, 16, 4, torch.bfloat16, True)
    logits = torch.randn(10, 16, generator=torch.Generator().manual_seed(8))
    ids, wt = run_route(logits, 4, norm=True)
    rid, rw = ref_route(logits, 4, norm=True)
    assert torch.equal(ids, rid) and math.isclose(float(wt.sum()), 10.0, rel_tol=1e-5)
    check_moe((x, ids, wt, w1, s1, w2, s2))
