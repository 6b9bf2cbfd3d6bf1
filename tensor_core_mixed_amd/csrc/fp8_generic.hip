// Block-scaled 8-bit product for any alignment, leading dimension and size:
//
//     C[m][n] = epi(init + sum over blocks b of 128 k of
//                          (sa[b][m] * sb[b, n]) * P_b[m][n]),
//     P_b[m][n] = sum over the block's k of A[m][k] * B[n][k],
//
// a 64 x 64 tile a workgroup, 4 x 4 outputs a thread, operands decoded to
// binary32 on their way to LDS one byte at a time (8192^3 21.5 ms, 51 TFLOP/s on
// the vector ALU; it serves what the tiles do not take).  The fast kernels keep
// this order: a block's sum first, in binary32, then one multiply-add with
// the product of its two scales.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace {

constexpr int kT = 64, kKC = 32;  // tile edge, k per LDS step (a divisor of the scale block)

__global__ __launch_bounds__(256) void fp8_generic_kernel(Fp8Args a, int64_t tiles_n) {
    __shared__ float la[kKC][kT + 4], lb[kKC][kT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kT, n0 = (int64_t)(blockIdx.x % tiles_n) * kT;
    float acc[4][4], p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
            float v = 0.f;
            if (m < a.M && n < a.N) {
                if (a.accum) v = load_c_any((const char*)a.C + (m * a.ldc + n) * c_elem_bytes(a.c_type), a.c_type);
                if (a.has_bias) v += load_float<F32>((const char*)a.bias, n);
            }
            acc[i][j] = v;
            p[i][j] = 0.f;
        }
    for (int64_t k0 = 0; k0 < a.K; k0 += kKC) {
        for (int e = tid; e < kKC * kT; e += 256) {
            const int kk = e % kKC, r = e / kKC;
            const int64_t k = k0 + kk;
            la[kk][r] = k < a.K && m0 + r < a.M ? fp8_decode(a.A[(m0 + r) * a.lda + k], a.a_e5m2) : 0.f;
            lb[kk][r] = k < a.K && n0 + r < a.N ? fp8_decode(a.B[(n0 + r) * a.ldb + k], a.b_e5m2) : 0.f;
        }
        __syncthreads();
#pragma unroll 4
        for (int kk = 0; kk < kKC; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) p[i][j] = __builtin_fmaf(la[kk][4 * ty + i], lb[kk][4 * tx + j], p[i][j]);
        __syncthreads();
        if ((k0 + kKC) % kScaleBlock == 0 || k0 + kKC >= a.K) {
            const int64_t b = k0 / kScaleBlock;
            float sm[4], sn[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + i;
                sm[i] = m < a.M ? load_float<F32>((const char*)a.sa, b * a.ldsa + m) : 0.f;
                sn[i] = n < a.N ? load_float<F32>((const char*)a.sb, a.b_row ? b * a.ldsb + n : n / kScaleBlock * a.ldsb + b) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = __builtin_fmaf(p[i][j], sm[i] * sn[j], acc[i][j]);
                    p[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
            if (m >= a.M || n >= a.N) continue;
            float v = acc[i][j];
            if (a.relu) v = v > 0.f ? v : 0.f;
            store_c_any((char*)a.C + (m * a.ldc + n) * c_elem_bytes(a.c_type), a.c_type, v);
        }
}

}  // namespace

int launch_fp8_generic(const Fp8Args& a, void* stream) {
    const int64_t tm = (a.M + kT - 1) / kT, tn = (a.N + kT - 1) / kT;
    hipLaunchKernelGGL(fp8_generic_kernel, dim3((unsigned)(tm * tn)), dim3(256), 0, (hipStream_t)stream, a, tn);
    return (int)hipGetLastError();
}

}  // namespace tcm
