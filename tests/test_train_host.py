"""The host side of the 4-bit product, its quantiser, the router's losses and gradient and the orthogonalised update, on
stand-ins for the HIP calls: launches of a call stay together, grids stay within a launch's limits, and what does not need
memory takes none."""
import pytest

import host_util

MUON = "(3.4445, -4.7750, 2.0315) * 5"
CALLS = {
    # launches, the call (p: addresses of the thread's own)
    "4-bit tiles": (2, """T.tcm_set_option("fp4_config", 2) or T.tcm_set_option("fp4_split", 2) or
                          T.tcm_gemm_mxfp4(300, 512, 1024, p(0), 512, p(1), 300, p(2), 512, p(3), 512, p(4), 512, T.TCM_MXFP4_F32, None, 0,
                                           None)"""),
    "4-bit few rows": (2, """T.tcm_set_option("fp4_config", 4) or T.tcm_set_option("fp4_split", 2) or
                             T.tcm_gemm_mxfp4(8, 512, 1024, p(0), 512, p(1), 8, p(2), 512, p(3), 512, p(4), 512, T.TCM_MXFP4_F32, None, 0,
                                              None)"""),
    "losses": (2, "T.tcm_moe_balance(1000, 64, 4, p(0), 64, T.TCM_F32_F32, p(1), None, p(2), p(3), None)"),
    "update": (17, f"T.tcm_orthogonalize(1, 200, 300, p(0), 300, 0, p(1), 300, 0, T.TCM_F32_F32, {MUON}, 1e-7, 1.0, None)"),
    "update of few rows": (7, f"T.tcm_orthogonalize(1, 100, 200, p(0), 200, 0, p(1), 200, 0, T.TCM_F32_F32, {MUON}, 1e-7, 1.0, None)"),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_of_a_call_stay_together(tmp_path, name):
    n, call = CALLS[name]
    host_util.run(tmp_path, f"""
        def call(p):
            return ({call})
        assert call(lambda i: at(10 + i)) == T.TCM_OK  # (the workspace grows)
        hip.stub_clear()
        mallocs = hip.stub_mallocs()
        assert call(lambda i: at(10 + i)) == T.TCM_OK
        assert hip.stub_mallocs() == mallocs
        per_call = len(launches())
        assert per_call == {n}, (per_call, T.tcm_last_plan())
        hip.stub_clear()
        hip.stub_pause(100)
        start = threading.Barrier(3)
        bad = []
        def run(t):
            start.wait()
            for _ in range(10):
                if call(lambda i: at(20 + 20 * t + i)) != T.TCM_OK:
                    bad.append(t)
        ts = [threading.Thread(target=run, args=(t,)) for t in range(3)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert not bad
        who = [l.thread for l in launches()]
        assert len(who) == 3 * 10 * per_call and len(set(who)) == 3
        for i in range(0, len(who), per_call):
            assert len(set(who[i:i + per_call])) == 1
    """)


@pytest.mark.parametrize("name,call", [
    ("quantise", "T.tcm_quantize_mxfp4(300, 500, at(10), 500, T.TCM_F16_F32, at(11), 250, at(12), 300, at(13), 150, at(14), 500, None)"),
    ("back", "T.tcm_dequantize_mxfp4(300, 500, at(10), 250, at(11), 300, at(12), 500, T.TCM_F16_F32, None)"),
    ("product", "T.tcm_gemm_mxfp4(300, 512, 256, at(10), 128, at(11), 300, at(12), 128, at(13), 512, at(14), 512, T.TCM_MXFP4_F32, None, 0, None)"),
    ("losses", "T.tcm_moe_balance(128, 64, 4, at(10), 64, T.TCM_F32_F32, at(11), None, at(12), at(13), None)"),
    ("update", f"T.tcm_orthogonalize(7, 40, 256, at(10), 256, 10240, at(11), 256, 10240, T.TCM_F32_F32, {MUON}, 1e-7, 1.0, None)"),
    ("gradient", "T.tcm_moe_route_grad(5000, 64, 4, at(10), 64, T.TCM_F32_F32, 1.0, at(11), None, at(12), at(13), at(14), at(15), 64, None)"),
])
def test_calls_that_allocate_nothing(tmp_path, name, call):
    host_util.run(tmp_path, f"""
        assert {call} == T.TCM_OK
        assert len(launches()) == 1 and hip.stub_mallocs() == 0, T.tcm_last_plan()
    """)


CHECK = """
        assert launches()
        for l in launches():
            assert 0 < l.grid.x and l.grid.x * l.block.x < 1 << 32, (l.grid.x, l.block.x, T.tcm_last_plan())
            assert 0 < l.grid.y < 1 << 16 and l.grid.z == 1 and l.block.x <= 1024 and l.block.y == l.block.z == 1
"""


@pytest.mark.parametrize("rows,cols", [(1, (1 << 31) - 1), (200, (1 << 31) - 129), ((1 << 31) - 1, 5), ((1 << 31) - 1, 300), ((1 << 24) + 3, 1000)])
def test_quantiser_grids(tmp_path, rows, cols):
    tiles, row_units = -(-cols // 128) * -(-rows // 128), -(-cols // 256) * -(-rows // 8)
    out = host_util.run(tmp_path, f"""
        rows, cols = {rows}, {cols}
        half = lambda n: (n + 1) // 2
        assert T.tcm_quantize_mxfp4(rows, cols, at(10), cols, T.TCM_F16_F32, at(1 << 10), half(cols), at(1 << 11), rows, at(1 << 12), half(rows),
                                    at(1 << 13), cols, None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x * l.grid.y for l in launches()))
        hip.stub_clear()
        assert T.tcm_quantize_mxfp4(rows, cols, at(10), cols, T.TCM_F16_F32, at(1 << 10), half(cols), at(1 << 11), rows, None, 0, None, 0,
                                    None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x * l.grid.y for l in launches()))
        hip.stub_clear()
        assert T.tcm_dequantize_mxfp4(rows, cols, at(1 << 10), half(cols), at(1 << 11), rows, at(10), cols, T.TCM_F32_F32, None) == T.TCM_OK
        {CHECK}
        print(sum(l.grid.x * l.grid.y for l in launches()))
    """)
    assert [int(x) for x in out.split()] == [tiles, row_units, row_units]


@pytest.mark.parametrize("config", [-1, 0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("split", [0, 2, 64])
@pytest.mark.parametrize("M,N", [(1 << 17, 1 << 17), ((1 << 18) - 3, 1 << 16), (1 << 12, (1 << 21) - 16), (60, (1 << 27) - 16), (1 << 20, 1 << 16)])
def test_product_grids(tmp_path, config, split, M, N):
    host_util.run(tmp_path, f"""
        assert T.tcm_set_option("fp4_config", {config}) == T.tcm_set_option("fp4_split", {split}) == T.TCM_OK
        st = T.tcm_gemm_mxfp4({M}, {N}, 8192, at(10), 4096, at(1 << 10), {M}, at(1 << 11), 4096, at(1 << 12), {N}, at(1 << 13), {N},
                              T.TCM_MXFP4_F32 | T.TCM_C_BF16, None, 0, None)
        assert st == T.TCM_OK or st == T.TCM_ERR_NOT_SUPPORTED and not launches(), st
        if st == T.TCM_OK:
            {CHECK.strip().replace(chr(10), chr(10) + "    ")}
    """)


@pytest.mark.parametrize("tokens,experts,topk", [((1 << 31) - 1, 4, 0), ((1 << 30) + 5, 1, 1), (1 << 24, 1024, 64), (129, 1000, 3)])
def test_router_training_grids(tmp_path, tokens, experts, topk):
    host_util.run(tmp_path, f"""
        a = ({tokens}, {experts}, {topk}, at(1), {experts}, T.TCM_F16_F32)
        assert T.tcm_moe_balance(*a, at(1 << 10), None, at(1 << 11), at(1 << 12), None) == T.TCM_OK
        {CHECK}
        assert len(launches()) == 2
        assert T.tcm_moe_route_grad(*a, 1.0, at(1 << 10), None, at(1 << 13), at(1 << 11), at(1 << 12), at(1 << 14), {experts}, None) == T.TCM_OK
        {CHECK}
        assert len(launches()) == 3
    """)


@pytest.mark.parametrize("batch,rows,cols", [((1 << 31) - 1, 1, 1), (1 << 20, 64, 64), (1 << 20, 64, 600), (60000, 1024, 100), (100000, 300, 200), (3, 20000, 20000), (1, 1, (1 << 20) - 32),
                                             (40, 8192, 1024)])
def test_update_grids_and_parts(tmp_path, batch, rows, cols):
    """Many entries go in parts of a call; the workspace holds one part's (2 GiB of them, or one entry)."""
    out = host_util.run(tmp_path, f"""
        n = {rows} * {cols}
        assert T.tcm_orthogonalize({batch}, {rows}, {cols}, at(1), {cols}, n, at(1 << 12), {cols}, n, T.TCM_F16_F32, (1.5, -0.5, 0.0), 1e-7, 1.0,
                                   None) == T.TCM_OK
        {CHECK}
        assert hip.stub_mallocs() == (T.tcm_last_plan().split()[-1] != "chunks=1")
        print(T.tcm_last_plan().split("chunk=")[1].split()[0], sum(l.block.x == 256 and l.grid.x > 0 for l in launches()))
    """)
    chunk = int(out.split()[0])
    n, m = min(rows, cols), max(rows, cols)
    pad = lambda x: -(-x // 32) * 32
    entry = 4 * (n * pad(m) + 2 * m * pad(n) + 2 * n * pad(n))
    rows = 64 if n <= 64 else 128
    chunks = -(-m // (16384 // rows))
    if n <= 64 and m <= 8192 or n <= 128 and (m <= 128 or batch * chunks <= 256):  # (16384 values of X a chunk, two S; one chunk needs nothing)
        entry = (chunks > 1) * chunks * 4 * (16384 + 2 * rows * rows)
    assert 1 <= chunk <= batch and (chunk == 1 or chunk * entry <= 2 << 30)


@pytest.mark.parametrize("rows,cols", [((1 << 20) - 32, (1 << 20) - 32)])
def test_update_without_steps_of_a_large_matrix(tmp_path, rows, cols):
    host_util.run(tmp_path, f"""
        assert T.tcm_orthogonalize(1, {rows}, {cols}, at(1), {cols}, 0, at(1 << 12), {cols}, 0, T.TCM_F16_F32, (), 1e-7, 1.0, None) == T.TCM_OK
        {CHECK}
    """)


@pytest.mark.parametrize("coef,fits", [((2.0 ** 39, 0, 0) * 2, False), ((2.0 ** -40, 0, 0) * 2, False), ((2.0 ** 60, 0, 0), True), ((2.0 ** -60, 0, 0), True),
                                       ((0, 2.0 ** 80, 0), False), ((1, 0, 2.0 ** -81), False), ((2.0 ** 20, 0, 0) * 3, False), ((2.0 ** 15, 0, 0) * 3, True),
                                       ((3.4445, -4.775, 2.0315) * 20, True)])
def test_coefficients_that_leave_the_range(tmp_path, coef, fits):
    host_util.run(tmp_path, f"""
        for n in (20, 200):
            st = T.tcm_orthogonalize(1, n, 300, at(1), 300, 0, at(2), 300, 0, T.TCM_F32_F32, {coef}, 0.0, 1.0, None)
            assert st == (T.TCM_OK if {fits} else T.TCM_ERR_NOT_SUPPORTED), st
            assert bool(launches()) == {fits}
    """)
