// Block-scaled 4-bit product for any alignment, leading dimension and size:
//
//     C[m][n] = epi(init + sum over blocks b of 32 k of 2^(ea[b, m] + eb[b, n]) P_b[m][n]),
//     P_b[m][n] = sum over the block's k of A[m][k] * B[n][k],
//
// a 64 x 64 tile a workgroup, 4 x 4 outputs a thread, operands decoded to
// binary32 on their way to LDS one byte at a time.  P_b is a multiple of 1/4
// below 2^11: exact.  The two scales are added as exponents, so only the
// scaled block leaves binary32's range where it does.  It multiplies on the vector
// ALU (37 x 5120 x 8192: 857 us, 12 on the tiles): operands at 16 bytes are what
// is meant to be fast.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace {

constexpr int kT = 64;  // tile edge

__device__ __forceinline__ float e2m1(unsigned code) {
    // (doubled: 0 1 2 3 4 6 8 12, four bits each)
    const float v = 0.5f * (float)((0xc8643210u >> (4 * (code & 7))) & 15);
    return (code & 8) ? -v : v;
}

__global__ __launch_bounds__(256) void fp4_generic_kernel(Fp4Args a, int64_t tiles_n) {
    __shared__ float la[kMxBlock][kT + 4], lb[kMxBlock][kT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kT, n0 = (int64_t)(blockIdx.x % tiles_n) * kT;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int64_t k0 = 0; k0 < a.K; k0 += kMxBlock) {
        for (int e = tid; e < kMxBlock / 2 * kT; e += 256) {
            const int kk = 2 * (e & 15), r = e >> 4;
            const int64_t k = k0 + kk;
            const unsigned x = k < a.K && m0 + r < a.M ? a.A[(m0 + r) * a.lda + k / 2] : 0;
            const unsigned y = k < a.K && n0 + r < a.N ? a.B[(n0 + r) * a.ldb + k / 2] : 0;
            const bool two = k + 1 < a.K;
            la[kk][r] = e2m1(x);
            lb[kk][r] = e2m1(y);
            la[kk + 1][r] = two ? e2m1(x >> 4) : 0.f;
            lb[kk + 1][r] = two ? e2m1(y >> 4) : 0.f;
        }
        __syncthreads();
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) p[i][j] = 0.f;
#pragma unroll 4
        for (int kk = 0; kk < kMxBlock; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) p[i][j] = __builtin_fmaf(la[kk][4 * ty + i], lb[kk][4 * tx + j], p[i][j]);
        __syncthreads();
        const int64_t word = k0 / kMxWord;
        const int shift = 8 * (int)(k0 / kMxBlock % 4);
        int ea[4], eb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = min(m0 + 4 * ty + i, a.M - 1), n = min(n0 + 4 * tx + i, a.N - 1);
            ea[i] = (a.sa[word * a.ldsa + m] >> shift) & 255;
            eb[i] = (a.sb[word * a.ldsb + n] >> shift) & 255;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += ea[i] == 255 || eb[j] == 255 ? __builtin_nanf("") : ldexpf(p[i][j], ea[i] + eb[j] - 254);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
            if (m < a.M && n < a.N) store_epilogue(a, acc[i][j], m, n);
        }
}

}  // namespace

int launch_fp4_generic(const Fp4Args& a, void* stream) {
    const int64_t tm = (a.M + kT - 1) / kT, tn = (a.N + kT - 1) / kT;
    hipLaunchKernelGGL(fp4_generic_kernel, dim3((unsigned)(tm * tn)), dim3(256), 0, (hipStream_t)stream, a, tn);
    return (int)hipGetLastError();
}

}  // namespace tcm
