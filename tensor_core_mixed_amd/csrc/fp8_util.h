// Conversions between binary32, the 16-bit types and the two 8-bit floating
// formats (OCP e4m3 "fn" and e5m2, the ones gfx950 converts in hardware).
#pragma once
#include <hip/hip_runtime.h>

#include "lowp.h"
#include "tcm_internal.h"

namespace tcm {

template <bool E5M2>
__device__ __forceinline__ float fp8_decode(unsigned byte) {
    if constexpr (E5M2) return __builtin_amdgcn_cvt_f32_bf8((int)byte, 0);
    else return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}
__device__ __forceinline__ float fp8_decode(unsigned byte, int e5m2) {
    return e5m2 ? fp8_decode<true>(byte) : fp8_decode<false>(byte);
}
// four values to four bytes, the first lowest (round to nearest even)
template <bool E5M2>
__device__ __forceinline__ unsigned fp8_encode4(float a, float b, float c, float d) {
    int w = 0;
    if constexpr (E5M2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return (unsigned)w;
}

// eight bytes to eight binary16 values: exact, NaN and infinity kept (an e5m2
// byte is the upper half of the binary16 value)
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
template <bool E5M2>
__device__ __forceinline__ f16x8_t fp8_to_f16x8(int w0, int w1) {
    f16x2_t h[4];
    if constexpr (E5M2) {
        h[0] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm((unsigned)w0, (unsigned)w0, 0x010c000cu));
        h[1] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm((unsigned)w0, (unsigned)w0, 0x030c020cu));
        h[2] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm((unsigned)w1, (unsigned)w1, 0x010c000cu));
        h[3] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm((unsigned)w1, (unsigned)w1, 0x030c020cu));
    } else {
        h[0] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false));
        h[1] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true));
        h[2] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false));
        h[3] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true));
    }
    return __builtin_shufflevector(__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3), __builtin_shufflevector(h[2], h[3], 0, 1, 2, 3), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// element i of a 16- or 32-bit float array at any address
template <int XT>
__device__ __forceinline__ float load_float(const char* base, int64_t i) {
    if constexpr (XT == F32) {
        float v;
        __builtin_memcpy(&v, base + 4 * i, 4);
        return v;
    } else {
        unsigned short h;
        __builtin_memcpy(&h, base + 2 * i, 2);
        if constexpr (XT == F16) return (float)__builtin_bit_cast(_Float16, h);
        else return __builtin_bit_cast(float, (unsigned)h << 16);
    }
}

// C's element (its type per c_type) at any address
__device__ __forceinline__ float load_c_any(const char* p, int c_type) {
    if (c_type == C_ACC) return load_float<F32>(p, 0);
    return c_type == C_F16 ? load_float<F16>(p, 0) : load_float<BF16>(p, 0);
}
__device__ __forceinline__ void store_c_any(char* p, int c_type, float v) {
    if (c_type == C_ACC) {
        __builtin_memcpy(p, &v, 4);
    } else {  // rounded to nearest even
        const unsigned short h = c_type == C_F16 ? __builtin_bit_cast(unsigned short, (_Float16)v)
                                                 : __builtin_bit_cast(unsigned short, (__bf16)v);
        __builtin_memcpy(p, &h, 2);
    }
}

// one element of C from its sum: + bias, + C's contents, ReLU, rounded to C's type
__device__ __forceinline__ void store_epilogue(const Fp8Args& a, float v, int64_t m, int64_t n) {
    if (a.has_bias) v += load_float<F32>((const char*)a.bias, n);
    char* c = (char*)a.C + (m * a.ldc + n) * c_elem_bytes(a.c_type);
    if (a.accum) v += load_c_any(c, a.c_type);
    if (a.relu) v = v > 0.f ? v : 0.f;
    store_c_any(c, a.c_type, v);
}

}  // namespace tcm
