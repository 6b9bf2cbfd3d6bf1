"""tcm_last_plan on a host without memory: nothing is thrown out of a C entry."""
import subprocess

import host_util

NEW = """
#include <cstdlib>
#include <new>
static bool none;
extern "C" void no_memory(int on) { none = on; }
void* operator new(std::size_t n) {
    void* p = none ? nullptr : std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
"""


def test_text_of_a_plan_needs_no_memory(tmp_path):
    (tmp_path / "new.cpp").write_text(NEW)
    lib = tmp_path / "libnew.so"
    subprocess.run(["g++", "-shared", "-fPIC", str(tmp_path / "new.cpp"), "-o", str(lib)], check=True)
    out = host_util.run(tmp_path, f"""
        new = ctypes.CDLL({str(lib)!r}, mode=ctypes.RTLD_GLOBAL)
        L, buf = T.lib(), ctypes.create_string_buffer(256)
        for call in (lambda: T.tcm_quantize_fp8(5, 200, at(10), 200, T.TCM_F32_F32, at(11), 200, at(12), 5, None, 0, None, 0, None),
                     lambda: T.tcm_moe_route(3, 8, 2, at(10), 8, T.TCM_F32_F32, None, 1.0, at(11), at(12), None),
                     lambda: T.tcm_gemm_fp8(3, 40, 64, at(10), 64, at(11), 3, at(12), 64, at(13), 1, at(14), 40, T.TCM_E4M3_F32, None, 0, None),
                     lambda: T.tcm_moe(3, 64, 32, 4, 2, at(10), 64, at(11), at(12), at(13), None, at(14), None, at(15), 64,
                                       T.TCM_F16_F32 | T.TCM_C_F16, None)):
            assert call() == T.TCM_OK
            new.no_memory(1)
            n = L.tcm_last_plan(buf, 256)
            new.no_memory(0)
            print(buf.value.decode())
            assert n == len(buf.value) > 0 and L.tcm_last_plan(buf, 8) == n and len(buf.value) == 7
    """)
    assert [line.split()[0] for line in out.splitlines()] == ["kernel=quantize", "kernel=route", "kernel=fp8_skinny", "kernel=moe_tile"]
