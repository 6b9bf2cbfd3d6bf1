"""The training operators as a program uses them: one step through all of them, several host threads, two streams, graphs
of several calls that share a stream's workspace."""
import os
import sys
import threading

import pytest
import torch

import tensor_core_mixed_amd as T

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315) * 5


@pytest.mark.parametrize("args", [[], ["--tokens", "137", "--hidden", "320", "--inter", "200", "--experts", "9", "--topk", "3"]])
def test_example(args):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mxfp4_training
    e = mxfp4_training.main(args)
    # binary32 results of sums and exponentials; a bf16 one of a sum in binary32's accuracy: half a step of 2^-8, and 2^-16 of its own
    assert e["losses"] < 1e-5 and e["dlogits"] < 1e-5 and e["update"] < 2.0 ** -8 + 2.0 ** -16
    # A 4-bit value is off by a fifth of itself (a quarter where it saturates), or by 0.25 scales where it is small; a scale is
    # a fourth of its block's largest value or less, for normal values under 0.8 of their spread: 0.25 and 0.2 of the norm at
    # most, 0.33 together, and a product's norm carries both operands' shares.
    assert max(e["y"], e["dx"], e["dW"]) < 0.33 * 2 ** 0.5


def product_caller(seed, s, M):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, K = 256, 8192  # (k in several ranges)
    A, B = (torch.randint(0, 256, (r, K // 2), generator=gen, device="cuda", dtype=torch.uint8) for r in (M, N))
    sa, sb = (torch.full((K // 128, r), 0x7F7E807F, dtype=torch.int64, device="cuda").to(torch.int32) for r in (M, N))

    def call(out):
        return T.tcm_gemm_mxfp4(M, N, K, A.data_ptr(), K // 2, sa.data_ptr(), M, B.data_ptr(), K // 2, sb.data_ptr(), N, out.data_ptr(), N,
                                T.TCM_MXFP4_F32, None, 0, s)
    return call, lambda: torch.empty(M, N, device="cuda")


def losses_caller(seed, s, tokens):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E, k = 200, 4
    x = torch.randn(tokens, E, generator=gen, device="cuda")
    ids = torch.topk(x, k, dim=1)[1].int().contiguous()

    def call(out):
        return T.tcm_moe_balance(tokens, E, k, x.data_ptr(), E, T.TCM_F32_F32, ids.data_ptr(), None, out.data_ptr() + 8, out.data_ptr(), s)
    return call, lambda: torch.zeros(E + 3, device="cuda")


def update_caller(seed, s, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.randn(rows, cols, generator=gen, device="cuda")

    def call(out):
        return T.tcm_orthogonalize(1, rows, cols, g.data_ptr(), cols, 0, out.data_ptr(), cols, 0, T.TCM_F32_F32, MUON, 1e-7, 1.0, s)
    return call, lambda: torch.empty(rows, cols, device="cuda")


def callers(s):
    return [product_caller(0, s, 300), product_caller(1, s, 12), losses_caller(2, s, 3000), update_caller(3, s, 150, 400), update_caller(4, s, 300, 90)]


def alone(cs):
    out = []
    for call, new in cs:
        o = new()
        assert call(o) == T.TCM_OK
        torch.cuda.synchronize()
        out.append(o.clone())
    return out


@pytest.mark.parametrize("s", ["current", "per thread"])
def test_threads(s):
    s = torch.cuda.current_stream().cuda_stream if s == "current" else 2  # (hipStreamPerThread)
    cs = callers(s)
    want = alone(cs)
    got = [[new() for _ in range(20)] for _, new in cs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(cs))

    def run(i):
        start.wait()
        for o in got[i]:
            if cs[i][0](o) != T.TCM_OK:
                bad.append(i)
    ts = [threading.Thread(target=run, args=(i,)) for i in range(len(cs))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    torch.cuda.synchronize()
    assert not bad
    for w, os_ in zip(want, got):
        for o in os_:
            assert torch.equal(o, w)


def test_two_streams_at_once():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ca, cb = callers(a.cuda_stream), callers(b.cuda_stream)
    want = alone(ca)
    oa, ob = [new() for _, new in ca], [new() for _, new in cb]
    torch.cuda.synchronize()
    for _ in range(3):
        for (f, _), x, (g, _), y in zip(ca, oa, cb[::-1], ob[::-1]):
            assert f(x) == T.TCM_OK and g(y) == T.TCM_OK
    torch.cuda.synchronize()
    for w, x, y in zip(want, oa, ob):
        assert torch.equal(x, w) and torch.equal(y, w)


def test_two_graphs_share_a_workspace():
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    cs = callers(s.cuda_stream)
    want = alone(cs)
    outs = [new() for _, new in cs]
    graphs = []
    with torch.cuda.stream(s):
        for part in (slice(0, 3), slice(3, 5)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for (call, _), o in zip(cs[part], outs[part]):
                    assert call(o) == T.TCM_OK
            graphs.append(g)
        for turn in range(4):
            for o in outs:
                o.zero_()
            for g in graphs[::1 if turn % 2 else -1]:
                g.replay()
            again = [new() for _, new in cs]
            for (call, _), o in zip(cs, again):  # eager work on the same workspace, between the replays
                assert call(o) == T.TCM_OK
            torch.cuda.synchronize()
            for w, o, p in zip(want, outs, again):
                assert torch.equal(o, w) and torch.equal(p, w)


def test_a_capture_that_would_grow_the_workspace_is_refused():
    s = torch.cuda.Stream()
    g = torch.randn(400, 900, device="cuda")
    o = torch.empty_like(g)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            st = T.tcm_orthogonalize(1, 400, 900, g.data_ptr(), 900, 0, o.data_ptr(), 900, 0, T.TCM_F32_F32, MUON, 1e-7, 1.0, s.cuda_stream)
            o.zero_()
    assert st == T.TCM_ERR_NOT_SUPPORTED
