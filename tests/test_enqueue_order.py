"""Calls from several host threads on one stream: the launches of a call that hand data on through the stream's workspace
follow one another, with no other call's launches between them."""
import pytest

import host_util

CALLS = {
    # launches, the call (p: addresses of the thread's own)
    "moe": (3, """T.tcm_moe(4, 256, 128, 8, 2, p(0), 256, p(1), p(2), p(3), None, p(4), None, p(5), 256,
                            T.TCM_BF16_F32 | T.TCM_C_BF16, None)"""),
    "moe in chunks": (6, """T.tcm_moe(1000, 256, 128, 8, 2, p(0), 256, p(1), p(2), p(3), None, p(4), None, p(5), 256,
                                      T.TCM_BF16_F32 | T.TCM_C_BF16, None)"""),
    "moe on the kernels of any alignment": (2, """T.tcm_moe(4, 255, 127, 8, 2, p(0), 255, p(1), p(2), p(3), None, p(4), None, p(5), 255,
                                                            T.TCM_BF16_F32 | T.TCM_C_BF16, None)"""),
    "8-bit tiles": (2, """T.tcm_set_option("fp8_split", 2) or T.tcm_gemm_fp8(300, 512, 512, p(0), 512, p(1), 300, p(2), 512, p(3), 4, p(4),
                                                                             512, T.TCM_E4M3_F32, None, 0, None)"""),
    "8-bit few rows": (2, """T.tcm_set_option("fp8_split", 2) or T.tcm_set_option("fp8_config", 4) or
                             T.tcm_gemm_fp8(8, 512, 512, p(0), 512, p(1), 8, p(2), 512, p(3), 4, p(4), 512, T.TCM_E4M3_F32, None, 0, None)"""),
    "few rows": (2, """T.tcm_set_option("gemv", 2) or T.tcm_gemm(4, 4096, 4096, p(0), 4096, p(1), 4096, p(2), 4096, T.TCM_F16_F32, None,
                                                                 0, None)"""),
    "few rows in the fixed array": (2, """T.tcm_set_option("gemv", 2) or T.tcm_gemm_noalloc(4, 4096, 4096, p(0), 4096, p(1), 4096, p(2),
                                                                                           4096, T.TCM_F16_F32, None, 0, None)"""),
    "split tiles": (2, """T.tcm_set_option("sk_fixup", 2) or T.tcm_set_option("force_mode", 2) or T.tcm_set_option("gemv", 1) or
                          T.tcm_gemm(512, 512, 8192, p(0), 8192, p(1), 512, p(2), 512, T.TCM_F16_F32, None, 0, None)"""),
    "convolution": (2, """T.tcm_set_option("sk_fixup", 2) or T.tcm_set_option("force_mode", 2) or
                          T.tcm_conv2d(1, 16, 16, 512, 512, 3, 3, 1, 1, 1, 1, 1, 1, p(0), p(1), p(2), T.TCM_F16_F32, None, 0, None)"""),
    "group": (2, """T.tcm_set_option("sk_fixup", 2) or T.tcm_set_option("force_mode", 2) or
                    T.tcm_gemm_grouped([(256, 512, p(0), 8192, p(1), 512, p(2), 512, None)] * 1, 8192, T.TCM_F16_F32, 0, None)"""),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_of_a_call_stay_together(tmp_path, name):
    n, call = CALLS[name]
    host_util.run(tmp_path, f"""
        def call(p):
            return ({call})
        assert call(lambda i: at(10 + i)) == T.TCM_OK  # (the workspace grows)
        assert len(launches()) >= {n}, len(launches())
        hip.stub_clear()
        assert call(lambda i: at(10 + i)) == T.TCM_OK
        per_call = len(launches())
        assert per_call == {n}, (per_call, T.tcm_last_plan())
        hip.stub_clear()
        hip.stub_pause(300)
        start = threading.Barrier(3)
        bad = []
        def run(t):
            start.wait()
            for _ in range(15):
                if call(lambda i: at(20 + 20 * t + i)) != T.TCM_OK:
                    bad.append(t)
        ts = [threading.Thread(target=run, args=(t,)) for t in range(3)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert not bad
        who = [l.thread for l in launches()]
        assert len(who) == 3 * 15 * per_call and len(set(who)) == 3
        for i in range(0, len(who), per_call):
            assert len(set(who[i:i + per_call])) == 1, (i, [sorted(set(who)).index(w) for w in who])
    """)


def test_each_threads_own_default_stream_has_a_workspace_of_its_own(tmp_path):
    """One handle, hipStreamPerThread, names another stream in every thread: their work may overlap."""
    host_util.run(tmp_path, """
        per_thread = 2  # (the handle's value)
        def call(p=lambda i: at(10 + i)):
            return T.tcm_moe(4, 256, 128, 8, 2, p(0), 256, p(1), p(2), p(3), None, p(4), None, p(5), 256, T.TCM_BF16_F32 | T.TCM_C_BF16,
                             per_thread)
        assert call() == call() == T.TCM_OK and hip.stub_mallocs() == 1
        done, go = [], threading.Barrier(2)
        def run():
            done.append(call() == call() == T.TCM_OK)
            go.wait()  # (both threads live at once)
        ts = [threading.Thread(target=run) for _ in range(2)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert done == [True, True] and hip.stub_mallocs() == 3, hip.stub_mallocs()
        assert call() == T.TCM_OK and hip.stub_mallocs() == 3
    """)
