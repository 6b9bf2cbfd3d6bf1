// Shared by the kernels of the orthogonalised update (ortho.hip,
// ortho_small.hip).
#pragma once
#include <hip/hip_runtime.h>

#include "lowp.h"

namespace tcm {
namespace ortho {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));

// a value's two parts, the upper in the lower half of the word
__device__ __forceinline__ unsigned split(float v) {
    asm("" : "+v"(v));  // (v is rounded to binary32 here, for both parts alike, and not where it comes from an fma for one of them)
    const _Float16 hi = (_Float16)v, lo = (_Float16)(v - (float)hi);
    return __builtin_bit_cast(unsigned, h2_t{hi, lo});
}
__device__ __forceinline__ unsigned upper2(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ unsigned lower2(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// 1 / (|G| + eps) of an entry, the same in every thread
__device__ __forceinline__ double inverse_norm(const OrthoArgs& a, int64_t entry) {
    double s = 0;
    for (int i = threadIdx.x & 63; i < a.slices; i += 64) s += a.squares[entry * a.slices + i];
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    return 1 / (sqrt(s) + (double)a.eps);
}

}  // namespace ortho
}  // namespace tcm
