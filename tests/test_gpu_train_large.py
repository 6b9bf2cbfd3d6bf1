"""Offsets past 32 bits in the 4-bit product, its quantiser, the router's losses and gradient and the orthogonalised update."""
import pytest
import torch

import lowp_util as L
import mx_util as U
import tensor_core_mixed_amd as T
import test_gpu_route_train as R

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


def test_quantiser_and_product():
    rows, cols, N = 70000, 65536, 48  # 4.6e9 values, 2.3e9 bytes of them in 4 bits
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    for r in range(0, rows, 10000):
        x[r:r + 10000] = torch.randn(min(10000, rows - r), cols, generator=gen, device="cuda", dtype=torch.bfloat16)
    q, s = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda"), torch.zeros(cols // 128, rows, dtype=torch.int32, device="cuda")
    qt, st = torch.zeros(cols, -(-rows // 32) * 16, dtype=torch.uint8, device="cuda"), torch.zeros(-(-rows // 128), cols, dtype=torch.int32, device="cuda")
    assert T.tcm_quantize_mxfp4(rows, cols, x.data_ptr(), cols, T.TCM_BF16_F32, q.data_ptr(), q.stride(0), s.data_ptr(), rows, qt.data_ptr(),
                                qt.stride(0), st.data_ptr(), cols, stream()) == T.TCM_OK
    at = [0, 1, 32767, 65535, 65536, 69998, 69999]
    codes, e = U.quantize(x[at].cpu())
    assert torch.equal(q[at].cpu(), U.pack(codes, cols // 2)) and torch.equal(s[:, at].cpu(), U.scale_words(e, len(at)))
    at_t = [0, 40000, 65535]
    ct, et = U.quantize(x[:, at_t].t().cpu())
    assert torch.equal(qt[at_t].cpu(), U.pack(ct, qt.shape[1], 0)) and torch.equal(st[:, at_t].cpu(), U.scale_words(et, len(at_t)))
    back = torch.zeros_like(x)
    assert T.tcm_dequantize_mxfp4(rows, cols, q.data_ptr(), q.stride(0), s.data_ptr(), rows, back.data_ptr(), cols, T.TCM_BF16_F32,
                                  stream()) == T.TCM_OK
    assert torch.equal(back[at].cpu().double(), U.values(codes, e))
    del back, x
    b, eb = U.operand(torch.Generator().manual_seed(1), N, cols, 1)
    hb, hs = U.pack(b, cols // 2).cuda(), U.scale_words(eb, N).cuda()
    for config in (-1, 4, 5):
        T.tcm_set_option("fp4_config", config)
        try:
            C = torch.zeros(rows, N, device="cuda")
            assert T.tcm_gemm_mxfp4(rows, N, cols, q.data_ptr(), q.stride(0), s.data_ptr(), rows, hb.data_ptr(), cols // 2, hs.data_ptr(), N,
                                    C.data_ptr(), N, T.TCM_MXFP4_F32, None, 0, stream()) == T.TCM_OK
            torch.cuda.synchronize()
        finally:
            T.tcm_set_option("fp4_config", -1)
        ref, bound = U.gemm_ref(codes, e, b, eb)
        L.check_close(C[at].cpu(), ref, bound)


def test_losses_and_gradient():
    tokens, E, k = 4_500_000, 600, 2  # 2.7e9 logits
    x = torch.empty(tokens, E, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    share, z, step = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0, 300_000
    ids = torch.empty(tokens, k, dtype=torch.int32, device="cuda")
    for t in range(0, tokens, step):
        part = torch.randn(step, E, generator=gen, device="cuda").bfloat16()
        x[t:t + step] = part
        f = part.float()
        ids[t:t + step] = torch.topk(f, k, dim=1)[1].int()
        share += torch.softmax(f, 1).double().sum(0)
        z += float(torch.logsumexp(f, 1).double().square().sum())
    counts, losses = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    assert T.tcm_moe_balance(tokens, E, k, x.data_ptr(), E, T.TCM_BF16_F32, ids.data_ptr(), None, counts.data_ptr(), losses.data_ptr(),
                             stream()) == T.TCM_OK
    want = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(counts[:-1].long(), want) and int(counts[-1]) == tokens
    loss = E * float((want.double() / (tokens * k) * share / tokens).sum())
    # (a lane adds 4.5e6 / 2048 shares of one sign in binary32: half a step of 2^-24 each at most)
    assert abs(float(losses[0]) - loss) < 3000 * 2.0 ** -24 * loss and abs(float(losses[1]) - z / tokens) < 1e-5 * z / tokens
    D = torch.empty(tokens, E, dtype=torch.bfloat16, device="cuda")
    dw, dl = torch.randn(tokens, k, generator=gen, device="cuda"), torch.tensor([1.0 * tokens, 0.1 * tokens], device="cuda")
    assert T.tcm_moe_route_grad(tokens, E, k, x.data_ptr(), E, T.TCM_BF16_F32 | T.TCM_C_BF16, 1.0, ids.data_ptr(), None, dw.data_ptr(),
                                counts.data_ptr(), dl.data_ptr(), D.data_ptr(), E, stream()) == T.TCM_OK
    torch.cuda.synchronize()
    at = [0, 3_579_139, 3_579_140, tokens - 1]  # (2^31 values lie before the second)
    ref, bound = R.grad_ref(x[at].cpu(), ids[at].cpu(), None, False, False, dw[at].cpu(), counts.cpu(), dl.cpu(), 1.0)
    assert ((D[at].cpu().double() - ref).abs() <= bound + (ref.abs() + bound) * 2.0 ** -8).all()


def test_update_of_entries_far_apart():
    rows, cols, far = 60, 90, (1 << 31) + 1000
    G = torch.zeros(2 * far + rows * cols, dtype=torch.bfloat16, device="cuda")
    O = torch.zeros_like(G)
    small = torch.randn(3, rows, cols, device="cuda").bfloat16()
    for e in range(3):
        G[e * far:e * far + rows * cols] = small[e].flatten()
    coef = (3.4445, -4.7750, 2.0315) * 5
    assert T.tcm_orthogonalize(3, rows, cols, G.data_ptr(), cols, far, O.data_ptr(), cols, far, T.TCM_BF16_F32 | T.TCM_C_BF16, coef, 1e-7, 1.0,
                               stream()) == T.TCM_OK
    o = torch.zeros_like(small)
    assert T.tcm_orthogonalize(3, rows, cols, small.data_ptr(), cols, rows * cols, o.data_ptr(), cols, rows * cols, T.TCM_BF16_F32 | T.TCM_C_BF16,
                               coef, 1e-7, 1.0, stream()) == T.TCM_OK
    torch.cuda.synchronize()
    for e in range(3):
        assert torch.equal(O[e * far:e * far + rows * cols].view(rows, cols), o[e])
