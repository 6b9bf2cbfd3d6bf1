"""The block-scaled 8-bit product and its quantiser on the GPU against 64-bit references."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, E5M2, X_CODE, blocks, check_close, gemm_ref, half_step, padded, quantize

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ quantiser

def run_quantize(x, t, tile, out, ldx=None, shift=0):
    """x (CPU) through the library; x's rows at ldx, every pointer `shift` bytes off; returns CPU (q, s, qt, st)."""
    rows, cols = x.shape
    ldx = ldx or cols
    es = x.element_size()
    buf = torch.full((max(rows * ldx, 1) * es + 16,), 0xFF, dtype=torch.uint8)  # a NaN in every type
    xv = torch.full((rows, ldx), float("nan"), dtype=x.dtype)
    xv[:, :cols] = x
    buf[shift:shift + rows * ldx * es] = xv.view(torch.uint8).flatten()
    buf = buf.cuda()
    mk = lambda r, c: torch.full((r * (c + 5) + 16,), 0x55, dtype=torch.uint8, device="cuda")
    q, qt = mk(rows, cols), mk(cols, rows)
    ss = (blocks(rows), blocks(cols)) if tile else (blocks(cols), rows)
    ts = (blocks(cols), blocks(rows)) if tile else (blocks(rows), cols)
    s, st = (torch.full((a, b + 3), -7.0, device="cuda") for a, b in (ss, ts))
    code = X_CODE[x.dtype] | (T.TCM_Q_E5M2 if t == E5M2 else 0) | (T.TCM_BLOCK_TILE if tile else 0)
    a = (q.data_ptr() + shift, cols + 5, s.data_ptr(), s.shape[1]) if out != "cols" else (None, 0, None, 0)
    b = (qt.data_ptr() + shift, rows + 5, st.data_ptr(), st.shape[1]) if out != "rows" else (None, 0, None, 0)
    assert T.tcm_quantize_fp8(rows, cols, buf.data_ptr() + shift, ldx, code, *a, *b, stream()) == T.TCM_OK
    torch.cuda.synchronize()
    res = []
    for used, qq, sc, (r, c), sh in ((out != "cols", q, s, (rows, cols), ss), (out != "rows", qt, st, (cols, rows), ts)):
        qq, sc = qq.cpu(), sc.cpu()
        if not used:
            assert (qq == 0x55).all() and (sc == -7).all()
            res += [None, None]
            continue
        body = qq[shift:shift + r * (c + 5)].view(r, c + 5)
        assert (body[:, c:] == 0x55).all() and (qq[:shift] == 0x55).all(), "bytes past the rows were written"
        assert (sc[:, sh[1]:] == -7).all()
        res += [body[:, :c].contiguous().view(t).double(), sc[:, :sh[1]].contiguous()]
    return res


def check_quantize(x, t, tile, out, **kw):
    q, s, qt, st = run_quantize(x, t, tile, out, **kw)
    for got, gs, m in ((q, s, x), (qt, st, x.t().contiguous())):
        if got is None:
            continue
        ref, rs = quantize(m, t, tile)
        assert torch.equal(gs.isnan(), rs.isnan()) and torch.equal(gs.nan_to_num(-1.0), rs.nan_to_num(-1.0)), "scales"
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.nan_to_num(-1.0), ref.nan_to_num(-1.0)), "values"


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t", [E4M3, E5M2])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 129), (129, 1), (16, 512), (127, 128), (130, 255), (257, 384), (300, 77)])
def test_quantize(shape, dtype, t, tile):
    gen = torch.Generator().manual_seed(shape[0] * 1000 + shape[1])
    x = (torch.randn(shape, generator=gen) * torch.exp(torch.randn(shape[0], 1, generator=gen))).to(dtype)
    for out in ("rows", "cols", "both"):
        check_quantize(x, t, tile, out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,pad", [(0, 3), (2, 0), (1, 1), (4, 8), (8, 6)])
def test_quantize_any_alignment(dtype, shift, pad):
    x = torch.randn(131, 200, generator=torch.Generator().manual_seed(shift)).to(dtype)
    check_quantize(x, E4M3, False, "both", ldx=200 + pad, shift=shift)
    check_quantize(x, E5M2, True, "both", ldx=200 + pad, shift=shift)


@pytest.mark.parametrize("t", [E4M3, E5M2])
def test_quantize_ties_and_neighbours(t):
    """Quotients on the middle of two values, and one unit of binary32 to either side of it."""
    from lowp_util import values
    tab = values(t)
    mid = ((tab[1:] + tab[:-1]) / 2).float()
    for scale in (1.0, 0.75, 3.0 * 2.0 ** -20, 2.0 ** -126, 2.0 ** 100):
        v = (mid.double() * scale).float()
        v = torch.cat([v, torch.nextafter(v, torch.tensor(0.0)), torch.nextafter(v, torch.tensor(torch.inf))])
        rows = torch.zeros(blocks(len(v)) + (-(-len(v) // 127)), 128)
        for i in range(0, len(v), 127):
            part = v[i:i + 127]
            rows[i // 127, 1:1 + len(part)] = part * (1 - 2 * (torch.arange(len(part)) % 2))
        big = float(tab[-1])
        rows[:, 0] = torch.tensor(big * scale, dtype=torch.float64).float()
        check_quantize(rows, t, False, "both")
        check_quantize(rows, t, True, "both")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_quantize_exact_ratios(dtype):
    """Small whole numbers: many quotients fall on ties exactly."""
    gen = torch.Generator().manual_seed(5)
    x = torch.randint(-63, 64, (256, 256), generator=gen).to(dtype)
    for t in (E4M3, E5M2):
        check_quantize(x, t, False, "both")
        check_quantize(x, t, True, "both")


@pytest.mark.parametrize("tile", [False, True])
def test_quantize_zeros_infinities_nan(tile):
    x = torch.randn(260, 390, generator=torch.Generator().manual_seed(1))
    x[:, 128:256] = 0
    x[3, 5] = float("inf")
    x[130, 300] = float("nan")
    x[200, 10], x[201, 10] = float("-inf"), float("nan")
    x[258] = 1e-42  # below the normal range
    x[259] = torch.finfo(torch.float32).max
    for t in (E4M3, E5M2):
        check_quantize(x, t, tile, "both")


# ------------------------------------------------------------------ product

def run_gemm(M, N, K, ta=E4M3, tb=E4M3, c=torch.float32, b_row=False, bias=False, relu=False, accum=False, lda=None, ldb=None,
             ldc=None, shift=0, seed=0, edit=None):
    gen = torch.Generator().manual_seed(seed * 7919 + M * 31 + N * 17 + K)
    lda, ldb, ldc = lda or max(16, -(-K // 16) * 16), ldb or max(16, -(-K // 16) * 16), ldc or N
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    w = torch.randn(N, K, generator=gen) * max(K, 1) ** -0.5
    A, sa = quantize(x, ta, False) if K else (torch.zeros(M, 0), torch.zeros(0, M))
    B, sb = quantize(w, tb, not b_row) if K else (torch.zeros(N, 0), torch.zeros(0, N) if b_row else torch.zeros(blocks(N), 0))
    bv = torch.randn(N, generator=gen) if bias else None
    c_in = torch.randn(M, N, generator=gen).to(c) if accum else None
    if edit:
        edit(A, sa, B, sb)
    dev = lambda b: torch.cat([torch.zeros(shift, dtype=torch.uint8), b.flatten()]).cuda()
    Ad, Bd = dev(padded(A, lda, ta)), dev(padded(B, ldb, tb))
    sad, sbd = (torch.nn.functional.pad(s, (0, 2), value=float("nan")).contiguous().cuda() for s in (sa, sb))
    C = torch.full((M, ldc), float("nan"), dtype=c)
    if accum:
        C[:, :N] = c_in
    Cd = torch.cat([torch.zeros(16, dtype=c), C.flatten(), torch.full((16,), 3.0, dtype=c)]).cuda()
    bd = bv.cuda() if bias else None
    code = T.TCM_E4M3_F32 | (T.TCM_A_E5M2 if ta == E5M2 else 0) | (T.TCM_B_E5M2 if tb == E5M2 else 0)
    code |= {torch.float32: 0, torch.float16: T.TCM_C_F16, torch.bfloat16: T.TCM_C_BF16}[c] | (T.TCM_B_ROW_SCALES if b_row else 0)
    epi = (T.TCM_EPI_BIAS if bias else 0) | (T.TCM_EPI_RELU if relu else 0) | (T.TCM_EPI_ACCUM if accum else 0)
    st = T.tcm_gemm_fp8(M, N, K, Ad.data_ptr() + shift, lda, sad.data_ptr(), sad.shape[1], Bd.data_ptr() + shift, ldb, sbd.data_ptr(),
                        sbd.shape[1], Cd.data_ptr() + 16 * Cd.element_size(), ldc, code, bd.data_ptr() if bias else None, epi, stream())
    assert st == T.TCM_OK, T.tcm_status_string(st)
    torch.cuda.synchronize()
    out = Cd.cpu()
    assert (out[-16:] == 3).all()
    got = out[16:-16].view(M, ldc)
    assert got[:, N:].isnan().all(), "columns past N were written"
    ref, bound = gemm_ref(A, sa, B, sb, b_row, bv, c_in, relu)
    return got[:, :N], ref, bound + half_step(ref, c) * (1 + 2.0 ** -10) + 2.0 ** -126


def gemm_magnitude(M, N, K, ta, tb, b_row):
    """The sums of the magnitudes of run_gemm's products (seed 0)."""
    gen = torch.Generator().manual_seed(M * 31 + N * 17 + K)
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    w = torch.randn(N, K, generator=gen) * max(K, 1) ** -0.5
    (A, sa), (B, sb) = quantize(x, ta, False), quantize(w, tb, not b_row)
    return gemm_ref(A.abs(), sa, B.abs(), sb, b_row)[0]


def check_gemm(*a, **kw):
    got, ref, bound = run_gemm(*a, **kw)
    check_close(got, ref, bound)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (3, 16, 130), (16, 16, 2048), (17, 33, 500), (33, 256, 384), (48, 130, 1000),
                                   (64, 64, 64), (65, 512, 256), (100, 300, 129), (128, 128, 4096), (250, 260, 640), (256, 512, 127),
                                   (300, 1000, 513)])
@pytest.mark.parametrize("b_row", [False, True])
def test_gemm_sizes(M, N, K, b_row):
    check_gemm(M, N, K, b_row=b_row, bias=True)


@pytest.mark.parametrize("ta,tb", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("c", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 20, 40, 60, 200])
def test_gemm_types(ta, tb, c, M):
    for b_row in (False, True):
        check_gemm(M, 144, 400, ta, tb, c, b_row, bias=M == 20, relu=M == 40, accum=M == 60)


@pytest.mark.parametrize("M", [1, 13, 50, 150])
@pytest.mark.parametrize("epi", range(8))
def test_gemm_epilogue(M, epi):
    check_gemm(M, 160, 272, c=torch.bfloat16 if epi % 3 else torch.float32, bias=bool(epi & 1), relu=bool(epi & 2), accum=bool(epi & 4))


@pytest.mark.parametrize("M", [2, 40, 140])
def test_gemm_any_alignment(M):
    for kw in (dict(lda=301), dict(ldb=301), dict(ldc=203), dict(shift=1), dict(shift=8), dict(lda=320, ldb=336, ldc=224),
               dict(ldc=204, c=torch.float16), dict(ldc=201, c=torch.bfloat16)):
        check_gemm(M, 200, 300, **kw)
        check_gemm(M, 200, 300, b_row=True, bias=True, **kw)


@pytest.mark.parametrize("M", [1, 30, 100])
def test_gemm_no_k(M):
    check_gemm(M, 70, 0, bias=True)
    check_gemm(M, 70, 0, accum=True, relu=True)


@pytest.mark.parametrize("M", [1, 24, 63, 90, 260])
@pytest.mark.parametrize("b_row", [False, True])
def test_gemm_scale_range(M, b_row):
    """Neighbouring blocks whose scales differ by 2^100, and blocks of zeros at the least scale."""
    def edit(A, sa, B, sb):
        sa[0] *= 2.0 ** 50
        sa[1] = 2.0 ** -126
        sa[2] *= 2.0 ** -50
        A[:, 128:256] = 0
    check_gemm(M, 256, 600, b_row=b_row, edit=edit)


@pytest.mark.parametrize("M", [1, 24, 63, 90, 260])
def test_gemm_nan_stays_in_its_row(M):
    bad = M - 1

    def edit(A, sa, B, sb):
        sa[1, bad] = float("nan")
    got, ref, bound = run_gemm(M, 256, 600, edit=edit)
    assert got[bad].isnan().all()
    keep = [m for m in range(M) if m != bad]
    check_close(got[keep], ref[keep], bound[keep])


@pytest.fixture
def options():
    yield T.tcm_set_option
    T.tcm_set_option("fp8_config", -1)
    T.tcm_set_option("fp8_split", 0)


@pytest.mark.parametrize("config", [0, 1, 2, 3])
@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (64, 128, 128), (257, 129, 1283), (300, 520, 1000), (130, 300, 390)])
def test_gemm_every_tile(options, config, split, M, N, K):
    assert options("fp8_config", config) == T.TCM_OK and options("fp8_split", split) == T.TCM_OK
    for b_row in (False, True):
        for ta, tb, c in ((E4M3, E4M3, torch.float32), (E5M2, E4M3, torch.bfloat16), (E4M3, E5M2, torch.float16)):
            got, ref, bound = run_gemm(M, N, K, ta, tb, c, b_row, bias=True, accum=b_row)
            name = (("256x256", "256x128", "128x128", "64x128")[config] if config or c != torch.float32 else "x128")
            assert f"{name} " in T.tcm_last_plan() and f"split={min(split, blocks(K))}" in T.tcm_last_plan()
            # 16-bit C: products cut to 2^-13 of the largest of their eight before they are added, each by less than a
            # unit; the largest is about a third of the eight's magnitudes and the cuts average half a unit
            mag = 0 if c == torch.float32 else 2.0 ** -12 * gemm_magnitude(M, N, K, ta, tb, b_row)
            check_close(got, ref, bound + mag)


@pytest.mark.parametrize("split", [1, 2, 5])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (16, 33, 1024), (17, 50, 2050), (48, 128, 777), (64, 300, 1664), (150, 40, 1300)])
def test_gemm_few_rows_kernel(options, split, M, N, K):
    assert options("fp8_config", 4) == T.TCM_OK and options("fp8_split", split) == T.TCM_OK
    for b_row in (False, True):
        for ta, tb, c in ((E4M3, E4M3, torch.float32), (E5M2, E4M3, torch.bfloat16), (E4M3, E5M2, torch.float16), (E5M2, E5M2, torch.float32)):
            check_gemm(M, N, K, ta, tb, c, b_row, bias=True, relu=M == 17, accum=b_row)
            assert "fp8_skinny" in T.tcm_last_plan()


def test_training_products_from_quantised_operands():
    """y, dx and dW of a linear layer from one quantisation each of x, W and dy, against the same products in 64 bits."""
    gen = torch.Generator().manual_seed(11)
    tok, din, dout = 203, 320, 272
    x, w, dy = (torch.randn(s, generator=gen).to(torch.bfloat16) for s in ((tok, din), (dout, din), (tok, dout)))
    pad = lambda n: -(-n // 16) * 16
    # a layer keeps rows at multiples of 16 bytes, so that every product runs on the fast kernels
    h = {}
    for name, m, t, tile in (("x", x, E4M3, False), ("w", w, E4M3, True), ("dy", dy, E5M2, False)):
        r, c = m.shape
        q, qt = torch.empty(r, pad(c), dtype=t, device="cuda"), torch.empty(c, pad(r), dtype=t, device="cuda")
        s = torch.empty((blocks(r), blocks(c)) if tile else (blocks(c), r), device="cuda")
        st = torch.empty((blocks(c), blocks(r)) if tile else (blocks(r), c), device="cuda")
        code = T.TCM_BF16_F32 | (T.TCM_Q_E5M2 if t == E5M2 else 0) | (T.TCM_BLOCK_TILE if tile else 0)
        md = m.cuda()
        assert T.tcm_quantize_fp8(r, c, md.data_ptr(), c, code, q.data_ptr(), q.stride(0), s.data_ptr(), s.shape[1], qt.data_ptr(),
                                  qt.stride(0), st.data_ptr(), st.shape[1], stream()) == T.TCM_OK
        h[name] = (q, s, qt, st)

    def product(M, N, K, A, sa, B, sb, flags):
        C = torch.empty(M, N, device="cuda")
        assert T.tcm_gemm_fp8(M, N, K, A.data_ptr(), A.stride(0), sa.data_ptr(), sa.shape[1], B.data_ptr(), B.stride(0), sb.data_ptr(),
                              sb.shape[1], C.data_ptr(), N, T.TCM_E4M3_F32 | flags, None, 0, stream()) == T.TCM_OK
        ref, bound = gemm_ref(A.cpu()[:, :K].double(), sa.cpu(), B.cpu()[:, :K].double(), sb.cpu(), bool(flags & T.TCM_B_ROW_SCALES))
        check_close(C.cpu(), ref, bound)
        return C.cpu().double()

    (xq, xs, xt, xst), (wq, ws, wt, wst), (gq, gs, gt, gst) = h["x"], h["w"], h["dy"]
    y = product(tok, dout, din, xq, xs, wq, ws, 0)
    dx = product(tok, din, dout, gq, gs, wt, wst, T.TCM_A_E5M2)
    dw = product(dout, din, tok, gt, gst, xt, xst, T.TCM_A_E5M2 | T.TCM_B_ROW_SCALES)
    # against unquantised products: every operand is off by half a step at most (2^-4, e5m2 2^-3, of its block's
    # values or of their smallest normal step), so an output by the sum of both shares of its magnitudes
    for got, a, b, ea, eb in ((y, x, w.t(), 2.0 ** -4, 2.0 ** -4), (dx, dy, w, 2.0 ** -3, 2.0 ** -4), (dw, dy.t(), x, 2.0 ** -3, 2.0 ** -4)):
        a, b = a.double(), b.double()
        # values under a type's normal range: off by up to half its least step, (largest / 2^15 for e4m3, 2^31 e5m2) of the block's
        mag = (a.abs() + a.abs().amax() * 2.0 ** -14) @ (b.abs() + b.abs().amax() * 2.0 ** -14)
        check_close(got, a @ b, mag * (ea + eb + ea * eb))


@pytest.mark.parametrize("M", [1, 40, 200, 500])
def test_gemm_repeats_and_graph(M):
    """The same bits from call to call, from a captured graph's replays, and on another stream."""
    N, K = 384, 2048
    gen = torch.Generator().manual_seed(3)
    A = torch.randn(M, K, generator=gen).to(E4M3).cuda()
    B = torch.randn(N, K, generator=gen).to(E4M3).cuda()
    sa, sb = torch.rand(blocks(K), M, generator=gen).cuda(), torch.rand(blocks(N), blocks(K), generator=gen).cuda()

    def call(C):
        assert T.tcm_gemm_fp8(M, N, K, A.data_ptr(), K, sa.data_ptr(), M, B.data_ptr(), K, sb.data_ptr(), blocks(K), C.data_ptr(), N,
                              T.TCM_E4M3_F32, None, 0, stream()) == T.TCM_OK
    first = torch.empty(M, N, device="cuda")
    call(first)
    C = torch.empty_like(first)
    for _ in range(3):
        C.zero_()
        call(C)
        assert torch.equal(C, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        C.zero_()
        call(C)
        s.synchronize()
        assert torch.equal(C, first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(C)
        for _ in range(3):
            C.zero_()
            g.replay()
            s.synchronize()
            assert torch.equal(C, first)
