"""The sums of the 8-bit product with 16-bit C, whose own rounding is taken out of the way: the products are added to a C
that holds their exact value rounded, so that what is left is small and keeps its bits."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, E5M2, blocks, check_close, gemm_ref, half_step, padded

pytestmark = pytest.mark.gpu


@pytest.fixture
def options():
    yield T.tcm_set_option
    T.tcm_set_option("fp8_config", -1)
    T.tcm_set_option("fp8_split", 0)


def check_sums(A, B, ta, tb, c, share):
    """A (M, K) and B (N, K) hold values of their types; unit scales.  Off by `share` of the sum of the products' magnitudes,
    what binary32 sums lose, and the rounding of what is left."""
    (M, K), N = A.shape, B.shape[0]
    sa, sb = torch.ones(blocks(K), M), torch.ones(blocks(N), blocks(K))
    ref, bound = gemm_ref(A, sa, B, sb, False)
    mag = A.double().abs() @ B.double().abs().t()
    c_in = (-ref).to(c)
    left = ref + c_in.double()
    assert left.isfinite().all()
    ld = -(-K // 16) * 16
    Ad, Bd, C, sad, sbd = padded(A, ld, ta).cuda(), padded(B, ld, tb).cuda(), c_in.cuda(), sa.cuda(), sb.cuda()
    code = T.TCM_E4M3_F32 | (T.TCM_A_E5M2 if ta == E5M2 else 0) | (T.TCM_B_E5M2 if tb == E5M2 else 0)
    code |= {torch.float32: 0, torch.float16: T.TCM_C_F16, torch.bfloat16: T.TCM_C_BF16}[c]
    assert T.tcm_gemm_fp8(M, N, K, Ad.data_ptr(), ld, sad.data_ptr(), M, Bd.data_ptr(), ld, sbd.data_ptr(), blocks(K), C.data_ptr(), N,
                          code, None, T.TCM_EPI_ACCUM, torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    # (2 * bound: binary32 sums, and their rounding on the way to what is left)
    total = share * mag + 2 * bound
    check_close(C.cpu(), left, total + half_step(left.abs() + total, c))


@pytest.mark.parametrize("config", [-1, 0, 1, 2, 3, 4])
@pytest.mark.parametrize("ta,tb", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("K", [128, 1000, 4096])
def test_normal_data(options, config, ta, tb, K):
    assert options("fp8_config", config) == T.TCM_OK
    gen = torch.Generator().manual_seed(K)
    A, B = torch.randn(130, K, generator=gen).to(ta).float(), torch.randn(150, K, generator=gen).to(tb).float()
    for c in (torch.float16, torch.bfloat16):
        check_sums(A, B, ta, tb, c, 2.0 ** -15)
    check_sums(A, B, ta, tb, torch.float32, 0)


@pytest.mark.parametrize("config", [-1, 0, 1, 2, 3, 4])
def test_small_products_next_to_large_ones(options, config):
    """One product in eight is 2^10 and the others fall below its thirteenth bit: seven of them, cut to nothing, are nearly
    2^-10 of the magnitudes.  Binary32 C holds them all."""
    assert options("fp8_config", config) == T.TCM_OK
    gen = torch.Generator().manual_seed(1)
    M, N, K = 130, 150, 512
    A, B = torch.full((M, K), 2.0 ** -4), torch.full((N, K), 1.875)
    large = torch.rand(K, generator=gen) < 1 / 8
    A[:, large], B[:, large] = 16.0, 64.0
    A *= 1 - 2.0 * (torch.rand(M, K, generator=gen) < 0.5)
    for c in (torch.float16, torch.bfloat16):
        check_sums(A, B, E4M3, E4M3, c, 2.0 ** -10)
    check_sums(A, B, E4M3, E4M3, torch.float32, 0)
    B[::2, large] = 448.0
    check_sums(A, B, E4M3, E4M3, torch.bfloat16, 2.0 ** -10)


@pytest.mark.parametrize("config", [-1, 0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("M", [9, 130])
@pytest.mark.parametrize("b_row", [False, True])
def test_scales_whose_product_is_subnormal(options, config, M, b_row):
    """Such a product is off by half the least step, 2^-150, which a block's sum multiplies."""
    assert options("fp8_config", config) == T.TCM_OK
    gen = torch.Generator().manual_seed(M)
    N, K = 150, 600
    A, B = (57344 * (2 * torch.rand(M, K, generator=gen) - 1)).to(E5M2).float(), (448 * (2 * torch.rand(N, K, generator=gen) - 1)).to(E4M3).float()
    power = lambda lo, hi, *s: 2.0 ** torch.randint(lo, hi, s, generator=gen) * (1 + torch.rand(s, generator=gen))
    sa, sb = power(-90, -74, blocks(K), M), power(-58, -50, *((blocks(K), N) if b_row else (blocks(N), blocks(K))))
    ref, bound = gemm_ref(A, sa, B, sb, b_row)
    bound = bound + 2.0 ** -150 * (A.double().abs() @ B.double().abs().t()) + 2.0 ** -149
    ld = -(-K // 16) * 16
    Ad, Bd, sad, sbd = padded(A, ld, E5M2).cuda(), padded(B, ld, E4M3).cuda(), sa.cuda(), sb.cuda()
    C = torch.full((M, N), 7.0, device="cuda")
    code = T.TCM_E4M3_F32 | T.TCM_A_E5M2 | (T.TCM_B_ROW_SCALES if b_row else 0)
    assert T.tcm_gemm_fp8(M, N, K, Ad.data_ptr(), ld, sad.data_ptr(), M, Bd.data_ptr(), ld, sbd.data_ptr(), sb.shape[1], C.data_ptr(), N,
                          code, None, 0, torch.cuda.current_stream().cuda_stream) == T.TCM_OK
    assert ref.abs().max() > 2.0 ** -120  # (ordinary numbers)
    check_close(C.cpu(), ref, bound)
