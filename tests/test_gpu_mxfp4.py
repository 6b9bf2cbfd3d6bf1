"""The 4-bit quantiser, its inverse and the product against references in 64 bits."""
import itertools

import pytest
import torch

import lowp_util as L
import mx_util as U
import tensor_core_mixed_amd as T

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]
OUT_FLAG = {torch.float32: 0, torch.float16: T.TCM_C_F16, torch.bfloat16: T.TCM_C_BF16}


def stream():
    return torch.cuda.current_stream().cuda_stream


def on_gpu(t, shift=0):
    """t's bytes on the GPU, `shift` bytes past an aligned address, as (holder, address)."""
    raw = t.contiguous().view(torch.uint8).flatten()
    buf = torch.empty(raw.numel() + 64, dtype=torch.uint8, device="cuda")
    buf[shift:shift + raw.numel()] = raw.cuda()
    return buf, buf.data_ptr() + shift


def back_from(buf, shift, like):
    n = like.numel() * like.element_size()
    return buf[shift:shift + n].clone().view(like.dtype).view(like.shape).cpu()


def run_quantize(x, out, pad=3, shift=0):
    """Both outputs' buffers after the call, filled with a pattern before it."""
    rows, cols = x.shape
    xb = torch.full((rows, cols + pad), 7.0, dtype=x.dtype)
    xb[:, :cols] = x
    hx, px = on_gpu(xb, shift * x.element_size())
    got = []
    args = []
    for r, c, on in ((rows, cols, out != "cols"), (cols, rows, out != "rows")):
        if not on:
            args += [None, 0, None, 0]
            got.append(None)
            continue
        q = torch.full((r, U.nbytes(c) + pad), 0xAA, dtype=torch.uint8)
        s = torch.full((U.words(c), r + pad), -1, dtype=torch.int32)
        (hq, pq), (hs, ps) = on_gpu(q, shift), on_gpu(s, 4 * shift)
        args += [pq, q.shape[1], ps, s.shape[1]]
        got.append((hq, q, hs, s))
    st = T.tcm_quantize_mxfp4(rows, cols, px, cols + pad, U.X_CODE[x.dtype], *args, stream())
    assert st == T.TCM_OK
    torch.cuda.synchronize()
    return [g and (back_from(g[0], shift, g[1]), back_from(g[2], 4 * shift, g[3])) for g in got]


def check_quantize(x, out, pad=3, shift=0):
    for got, m in zip(run_quantize(x, out, pad, shift), (x, x.t())):
        if got is None:
            continue
        codes, e = U.quantize(m)
        assert torch.equal(got[0], U.pack(codes, got[0].shape[1]))
        assert torch.equal(got[1], U.scale_words(e, got[1].shape[1]))


def normal(gen, rows, cols, t):
    x = torch.randn(rows, cols, generator=gen) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=gen).float())
    return x.to(t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("out", ["rows", "cols", "both"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (33, 33), (7, 128), (127, 129), (128, 128), (130, 257), (300, 95),
                                       (31, 1000), (512, 640)])
def test_quantize(t, out, rows, cols):
    gen = torch.Generator().manual_seed(rows * 1000 + cols)
    check_quantize(normal(gen, rows, cols, t), out)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 1), (5, 3), (8, 0)])
def test_quantize_any_alignment(t, pad, shift):
    gen = torch.Generator().manual_seed(5)
    check_quantize(normal(gen, 140, 151, t), "both", pad, shift)


@pytest.mark.parametrize("t", TYPES)
def test_quantize_edges(t):
    """Middles of neighbouring values, values past 6, zero blocks, the type's least and largest values, NaN and infinities."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 6.5, 7, 7.5, 0.5, 4, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -7.9,
                        0, -0.0, 1, 2, 3, 0.24, 0.26, 4.9, 5.1, -6, 7.99])
    f = torch.finfo(t)
    rows = [mid.to(t)]
    rows += [(mid * 2.0 ** k).to(t) for k in (-10, 3, 9)]
    rows += [torch.zeros(32, dtype=t), torch.full((32,), f.max, dtype=t), -torch.full((32,), f.smallest_normal, dtype=t)]
    least = torch.zeros(32, dtype=t)
    least[3], least[5] = f.smallest_normal * f.eps, -f.smallest_normal * f.eps
    rows.append(least)
    for bad in (float("nan"), float("inf"), -float("inf")):
        r = mid.to(t).clone()
        r[17] = bad
        rows.append(r)
    x = torch.stack(rows)
    assert x.shape == (11, 32)
    check_quantize(x, "both")
    check_quantize(x.t().contiguous(), "both")
    check_quantize(x.repeat(13, 11), "both")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 31, 1, 1), (33, 33, 2, 3), (130, 257, 3, 0), (16, 512, 0, 0), (9, 7, 5, 1)])
def test_dequantize(t, rows, cols, pad, shift):
    gen = torch.Generator().manual_seed(cols)
    codes, e = U.operand(gen, rows, cols, 12)
    e[0, 0] = 255
    e[-1, 0] = 0 if t != torch.float16 else 127 - 26  # half of it is the least value but one that the type's subnormals can be off by
    hq, pq = on_gpu(U.pack(codes, U.nbytes(cols) + pad, 0xFF), shift)
    hs, ps = on_gpu(U.scale_words(e, rows + pad))
    x = torch.full((rows, cols + pad), 7.0, dtype=t)
    hx, px = on_gpu(x, shift * x.element_size())
    assert T.tcm_dequantize_mxfp4(rows, cols, pq, U.nbytes(cols) + pad, ps, rows + pad, px, cols + pad, U.X_CODE[t], stream()) == T.TCM_OK
    torch.cuda.synchronize()
    got = back_from(hx, shift * x.element_size(), x)
    want = U.values(codes, e).float().to(t)  # (the values are exact in float32)
    assert torch.equal(got[:, :cols].isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got[:, :cols].float()), torch.nan_to_num(want.float()))
    assert (got[:, cols:] == 7).all()


def run_gemm(a, ea, b, eb, c_type, bias=None, c_in=None, relu=False, pad=(0, 0, 0), shift=0, align=16):
    """C (M, N) of one call; what lies past the rows' ends holds values and scales that must not be used."""
    M, K = a.shape
    N = b.shape[0]
    ld = -(-U.nbytes(max(K, 1)) // align) * align
    last = -(-K // 32)  # blocks past K: a scale of NaN
    ea, eb = ea.clone(), eb.clone()
    ea[:, last:] = eb[:, last:] = 255
    half = torch.zeros(M, 2 * ld, dtype=torch.uint8) + 15  # (an odd row's last half byte too)
    half[:, :K] = a
    qa = half[:, 0::2] | half[:, 1::2] << 4
    half = torch.zeros(N, 2 * ld, dtype=torch.uint8) + 15
    half[:, :K] = b
    qb = half[:, 0::2] | half[:, 1::2] << 4
    (ha, pa), (hb, pb) = on_gpu(qa, shift), on_gpu(qb, shift)
    (hsa, psa), (hsb, psb) = on_gpu(U.scale_words(ea, M + pad[0])), on_gpu(U.scale_words(eb, N + pad[1]))
    C = torch.full((M, N + pad[2]), 3.0, dtype=c_type)
    if c_in is not None:
        C[:, :N] = c_in
    hc, pc = on_gpu(C, shift * C.element_size())
    hbias = bias.cuda() if bias is not None else None
    epi = (T.TCM_EPI_BIAS if bias is not None else 0) | (T.TCM_EPI_ACCUM if c_in is not None else 0) | (T.TCM_EPI_RELU if relu else 0)
    st = T.tcm_gemm_mxfp4(M, N, K, pa, ld, psa, M + pad[0], pb, ld, psb, N + pad[1], pc, N + pad[2], T.TCM_MXFP4_F32 | OUT_FLAG[c_type],
                          hbias.data_ptr() if bias is not None else None, epi, stream())
    assert st == T.TCM_OK, (st, T.tcm_last_plan())
    torch.cuda.synchronize()
    got = back_from(hc, shift * C.element_size(), C)
    assert (got[:, N:] == 3).all()
    return got[:, :N]


def check_gemm(M, N, K, c_type, bias=False, accum=False, relu=False, spread=3, seed=0, **kw):
    gen = torch.Generator().manual_seed(seed + M + 7 * N + 49 * K)
    a, ea = U.operand(gen, M, K, spread)
    b, eb = U.operand(gen, N, K, spread)
    v = torch.randn(N, generator=gen) if bias else None
    c = torch.randn(M, N, generator=gen).to(c_type) if accum else None
    ref, bound = U.gemm_ref(a, ea, b, eb, v, c, relu)
    got = run_gemm(a, ea, b, eb, c_type, v, c, relu, **kw)
    L.check_close(got, ref, bound * 1.01 + L.half_step(ref.abs() + bound, c_type))
    return T.tcm_last_plan()


SIZES = [(1, 1, 1), (1, 16, 31), (3, 5, 32), (16, 17, 33), (5, 130, 127), (17, 64, 128), (64, 64, 129), (33, 70, 255), (65, 129, 256),
         (100, 200, 257), (127, 300, 384), (130, 33, 511), (64, 260, 513), (2, 3, 1000)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("c_type", TYPES)
def test_gemm(M, N, K, c_type):
    check_gemm(M, N, K, c_type, bias=K % 2 == 1, relu=M % 2 == 0)


class forced:
    def __init__(self, **options):
        self.options = options

    def __enter__(self):
        for k, v in self.options.items():
            assert T.tcm_set_option(k, v) == T.TCM_OK

    def __exit__(self, *_):
        for k in self.options:
            T.tcm_set_option(k, -1 if k.endswith("config") else 0)


KERNELS = {0: "tile=256x256", 1: "tile=256x128", 2: "tile=128x128", 3: "tile=64x128", 4: "fp4_skinny", 5: "fp4_generic"}


@pytest.mark.parametrize("config", list(KERNELS))
@pytest.mark.parametrize("M,N,K", SIZES + [(300, 520, 1024), (257, 513, 1281), (512, 256, 2304)])
@pytest.mark.parametrize("c_type", [torch.float32, torch.bfloat16])
def test_gemm_every_kernel(config, M, N, K, c_type):
    with forced(fp4_config=config):
        assert KERNELS[config] in check_gemm(M, N, K, c_type, bias=True, accum=K % 2 == 0, pad=(1, 2, 8 if M % 2 else 5))


@pytest.mark.parametrize("config", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("split", [2, 3, 7, 64])
@pytest.mark.parametrize("M,N,K", [(33, 70, 255), (65, 129, 1300), (300, 260, 2049), (20, 50, 20000)])
@pytest.mark.parametrize("c_type", [torch.float32, torch.float16])
def test_gemm_split(config, split, M, N, K, c_type):
    with forced(fp4_config=config, fp4_split=split):
        plan = check_gemm(M, N, K, c_type, bias=True, accum=True, relu=True)
        assert KERNELS[config] in plan and f"split={min(split, -(-K // 256))} " in plan


@pytest.mark.parametrize("config", [0, 1, 2, 3, 4])
def test_gemm_nan_scales_of_every_kernel(config):
    with forced(fp4_config=config):
        test_gemm_nan_scales()
        test_gemm_scales_of_the_whole_range()


@pytest.mark.parametrize("shift,align,pad", [(1, 1, (1, 2, 3)), (0, 1, (0, 0, 0)), (8, 8, (3, 0, 1)), (0, 16, (5, 1, 1))])
@pytest.mark.parametrize("c_type", TYPES)
def test_gemm_any_alignment(shift, align, pad, c_type):
    check_gemm(70, 90, 301, c_type, bias=True, accum=True, shift=shift, align=align, pad=pad)


@pytest.mark.parametrize("c_type", TYPES)
@pytest.mark.parametrize("bias,accum,relu", list(itertools.product([False, True], repeat=3)))
def test_gemm_epilogues(c_type, bias, accum, relu):
    check_gemm(40, 72, 200, c_type, bias, accum, relu)


def test_gemm_of_no_k():
    bias = torch.arange(5.0)
    z = torch.zeros(3, 0, dtype=torch.uint8)
    got = run_gemm(z, torch.zeros(3, 0, dtype=torch.int64), torch.zeros(5, 0, dtype=torch.uint8), torch.zeros(5, 0, dtype=torch.int64),
                   torch.float32, bias)
    assert torch.equal(got, bias.expand(3, 5))


def test_gemm_nan_scales():
    gen = torch.Generator().manual_seed(1)
    a, ea = U.operand(gen, 40, 300, 2)
    b, eb = U.operand(gen, 50, 300, 2)
    ea[7, 3], eb[11, 9] = 255, 255
    ref, bound = U.gemm_ref(a, ea, b, eb)
    got = run_gemm(a, ea, b, eb, torch.float32)
    assert torch.equal(got.isnan(), ref.isnan()) and ref.isnan().sum() == 40 + 50 - 1
    L.check_close(torch.nan_to_num(got), torch.nan_to_num(ref), torch.nan_to_num(bound))


def test_gemm_scales_of_the_whole_range():
    """Scales whose sum is an ordinary exponent though each lies far outside."""
    gen = torch.Generator().manual_seed(2)
    a, ea = U.operand(gen, 33, 200, 1)
    b, eb = U.operand(gen, 47, 200, 1)
    ea += 110
    eb -= 110
    ref, bound = U.gemm_ref(a, ea, b, eb)
    L.check_close(run_gemm(a, ea, b, eb, torch.float32), ref, bound)


def test_gemm_follows_the_quantiser():
    """A training step's three products from one quantisation each of x, w and dy."""
    gen = torch.Generator().manual_seed(3)
    tok, din, dout = 75, 160, 97
    m = {"x": torch.randn(tok, din, generator=gen), "w": torch.randn(dout, din, generator=gen), "g": torch.randn(tok, dout, generator=gen)}
    q = {}
    for name, v in m.items():
        r, c = v.shape
        q[name] = [torch.zeros(r, -(-c // 32) * 16, dtype=torch.uint8, device="cuda"), torch.zeros(U.words(c), r, dtype=torch.int32, device="cuda"),
                   torch.zeros(c, -(-r // 32) * 16, dtype=torch.uint8, device="cuda"), torch.zeros(U.words(r), c, dtype=torch.int32, device="cuda")]
        d = v.cuda()
        a = q[name]
        assert T.tcm_quantize_mxfp4(r, c, d.data_ptr(), c, T.TCM_F32_F32, a[0].data_ptr(), a[0].stride(0), a[1].data_ptr(), r,
                                    a[2].data_ptr(), a[2].stride(0), a[3].data_ptr(), c, stream()) == T.TCM_OK
    def product(M, N, K, a, sa, b, sb):
        C = torch.zeros(M, N, device="cuda")
        assert T.tcm_gemm_mxfp4(M, N, K, a.data_ptr(), a.stride(0), sa.data_ptr(), M, b.data_ptr(), b.stride(0), sb.data_ptr(), N,
                                C.data_ptr(), N, T.TCM_MXFP4_F32, None, 0, stream()) == T.TCM_OK
        return C.cpu()
    x, w, g = q["x"], q["w"], q["g"]
    for got, a, b in ((product(tok, dout, din, x[0], x[1], w[0], w[1]), m["x"], m["w"]),
                      (product(tok, din, dout, g[0], g[1], w[2], w[3]), m["g"], m["w"].t()),
                      (product(dout, din, tok, g[2], g[3], x[2], x[3]), m["g"].t(), m["x"].t())):
        ref, bound = U.gemm_ref(*U.quantize(a), *U.quantize(b))
        L.check_close(got, ref, bound)
