"""Host threads that call on one stream at once: every call gives the bits that it gives alone."""
import threading

import pytest
import torch

import tensor_core_mixed_amd as T
from lowp_util import E4M3, blocks

pytestmark = pytest.mark.gpu


def moe_caller(seed, stream):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tok, H, I, E, k = 12, 512, 256, 8, 4
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, w1, w2 = rnd(tok, H).bfloat16(), (rnd(E, 2, I, H) * H ** -0.5).bfloat16(), (rnd(E, H, I) * I ** -0.5).bfloat16()
    wt, ids = torch.topk(torch.rand(tok, E, generator=gen, device="cuda"), k, dim=1)
    ids = ids.int().contiguous()

    def call(out):
        return T.tcm_moe(tok, H, I, E, k, x.data_ptr(), H, ids.data_ptr(), wt.data_ptr(), w1.data_ptr(), None, w2.data_ptr(), None,
                         out.data_ptr(), H, T.TCM_BF16_F32 | T.TCM_C_BF16, stream)
    return call, lambda: torch.empty(tok, H, dtype=torch.bfloat16, device="cuda")


def product_caller(seed, stream, M):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, K = 256, 4096  # (k in several ranges)
    A, B = (torch.randn(r, K, generator=gen, device="cuda").to(E4M3) for r in (M, N))
    sa, sb = torch.rand(blocks(K), M, generator=gen, device="cuda"), torch.rand(blocks(N), blocks(K), generator=gen, device="cuda")

    def call(out):
        return T.tcm_gemm_fp8(M, N, K, A.data_ptr(), K, sa.data_ptr(), M, B.data_ptr(), K, sb.data_ptr(), blocks(K), out.data_ptr(), N,
                              T.TCM_E4M3_F32, None, 0, stream)
    return call, lambda: torch.empty(M, N, device="cuda")


def few_rows_caller(seed, stream):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, N, K = 3, 512, 8192
    A, B = (torch.randn(*s, generator=gen, device="cuda").half() for s in ((M, K), (K, N)))

    def call(out):
        return T.tcm_gemm(M, N, K, A.data_ptr(), K, B.data_ptr(), N, out.data_ptr(), N, T.TCM_F16_F32, None, 0, stream)
    return call, lambda: torch.empty(M, N, device="cuda")


def test_threads_on_one_stream():
    check_threads(torch.cuda.current_stream().cuda_stream)


def test_threads_on_their_own_default_streams():
    check_threads(2)  # (hipStreamPerThread, one handle for a stream of each thread)


def check_threads(s):
    callers = [moe_caller(0, s), moe_caller(1, s), product_caller(2, s, 300), product_caller(3, s, 40), few_rows_caller(4, s)]
    alone = []
    for call, new in callers:
        alone.append(new())
        assert call(alone[-1]) == T.TCM_OK
    outs = [[new() for _ in range(40)] for _, new in callers]
    torch.cuda.synchronize()
    status, start = [], threading.Barrier(len(callers))

    def run(call, mine):
        start.wait()
        status.extend(call(o) for o in mine)
    threads = [threading.Thread(target=run, args=(call, mine)) for (call, _), mine in zip(callers, outs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert len(status) == 40 * len(callers) and set(status) == {T.TCM_OK}
    for a, mine in zip(alone, outs):
        assert all(torch.equal(o, a) for o in mine)
