"""Offsets past 32 bits in the 8-bit product, its quantiser and the expert layer."""
import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, blocks, check_close, gemm_ref, half_step, moe_ref, quantize

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("c", [torch.float32, torch.bfloat16])
def test_gemm_far_rows(c):
    M, N, K, lda, ldc = 66000, 128, 250, 65536, 66000
    gen = torch.Generator().manual_seed(0)
    at = torch.cat([torch.arange(70), torch.arange(32750, 32820), torch.arange(M - 70, M)])  # rows with values, the others zeros
    x = torch.randn(len(at), K, generator=gen)
    q, s = quantize(x, E4M3, False)
    B, sb = quantize(torch.randn(N, K, generator=gen) * K ** -0.5, E4M3, True)
    A = torch.zeros(M, lda, dtype=torch.uint8, device="cuda")
    A[at.cuda(), :K] = q.to(E4M3).view(torch.uint8).cuda()
    sa = torch.zeros(blocks(K), M)
    sa[:, at] = s
    sa, sbd, Bd = sa.cuda(), sb.cuda(), torch.nn.functional.pad(B, (0, 6)).to(E4M3).cuda()
    C = torch.full((M, ldc), 7.0, dtype=c, device="cuda")
    code = T.TCM_E4M3_F32 | (T.TCM_C_BF16 if c == torch.bfloat16 else 0)
    assert T.tcm_gemm_fp8(M, N, K, A.data_ptr(), lda, sa.data_ptr(), M, Bd.data_ptr(), 256, sbd.data_ptr(), blocks(K), C.data_ptr(), ldc,
                          code, None, 0, stream()) == T.TCM_OK
    assert "fp8_tile" in T.tcm_last_plan()
    ref, bound = gemm_ref(q, s, B, sb, False)
    # 16-bit C: products cut to 2^-13 of the largest of their eight (see the tiles' own tests)
    mag = 0 if c == torch.float32 else 2.0 ** -12 * gemm_ref(q.abs(), s, B.abs(), sb, False)[0]
    check_close(C[at.cuda(), :N].cpu(), ref, bound + mag + half_step(ref, c) * (1 + 2.0 ** -10) + 2.0 ** -126)
    assert (C[:, N:N + 8] == 7).all() and (C[5000:5100, :N] == 0).all()


def test_quantize_far_rows():
    rows, cols, ldx, ldq = 66000, 200, 33000, 66000
    gen = torch.Generator().manual_seed(1)
    at = torch.cat([torch.arange(128), torch.arange(rows - rows % 128 - 128, rows)])
    x = torch.randn(len(at), cols, generator=gen).bfloat16()
    X = torch.zeros(rows, ldx, dtype=torch.bfloat16, device="cuda")
    X[at.cuda(), :cols] = x.cuda()
    Q = torch.full((rows, ldq), 0x55, dtype=torch.uint8, device="cuda")
    QT = torch.zeros(cols, rows, dtype=torch.uint8, device="cuda")
    S, ST = torch.zeros(blocks(cols), rows, device="cuda"), torch.zeros(blocks(rows), cols, device="cuda")
    assert T.tcm_quantize_fp8(rows, cols, X.data_ptr(), ldx, T.TCM_BF16_F32, Q.data_ptr(), ldq, S.data_ptr(), rows, QT.data_ptr(), rows,
                              ST.data_ptr(), cols, stream()) == T.TCM_OK
    ref, rs = quantize(x, E4M3, False)
    assert torch.equal(Q[at.cuda(), :cols].cpu().view(E4M3).double(), ref) and torch.equal(S[:, at.cuda()].cpu(), rs)
    assert (Q[:, cols:cols + 8] == 0x55).all()
    last = x[128:]  # the last two row blocks, the second of them partial
    ref, rs = quantize(last.t().contiguous(), E4M3, False)
    assert torch.equal(QT[:, rows - len(last):].cpu().view(E4M3).double(), ref) and torch.equal(ST[-2:].cpu(), rs)


def test_moe_far_experts():
    E, H, I, tok = 520, 2048, 1024, 3  # 4.4 GB of the first matrix
    gen = torch.Generator().manual_seed(2)
    far = [0, 300, E - 1]
    x = torch.randn(tok, H, generator=gen).bfloat16()
    w1, w2 = (torch.randn(3, 2, I, H, generator=gen) * H ** -0.5).bfloat16(), (torch.randn(3, H, I, generator=gen) * I ** -0.5).bfloat16()
    ids = torch.tensor([[0, 1], [2, 0], [1, 2]], dtype=torch.int32)
    wt = torch.rand(tok, 2, generator=gen)
    W1 = torch.empty(E, 2, I, H, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))  # experts that no token chose are not read
    W2 = torch.empty(E, H, I, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    for j, e in enumerate(far):
        W1[e], W2[e] = w1[j].cuda(), w2[j].cuda()
    idd = torch.tensor(far, dtype=torch.int32)[ids.long()].cuda()
    xd, wd, out = x.cuda(), wt.cuda(), torch.empty(tok, H, dtype=torch.bfloat16, device="cuda")
    assert T.tcm_moe(tok, H, I, E, 2, xd.data_ptr(), H, idd.data_ptr(), wd.data_ptr(), W1.data_ptr(), None, W2.data_ptr(), None,
                     out.data_ptr(), H, T.TCM_BF16_F32 | T.TCM_C_BF16, stream()) == T.TCM_OK
    assert "moe_tile" in T.tcm_last_plan()
    ref, bound = moe_ref(x, ids, wt, w1, None, w2, None)
    check_close(out.cpu(), ref, bound + half_step(ref, torch.bfloat16) * (1 + 2.0 ** -10) + 2.0 ** -126)
