// Block-scaled 4-bit product of a few rows (a decoding batch): B is read once
// and binds the time, so its bytes go straight from memory to registers.
//
// A workgroup takes 16 columns and up to 64 rows; its eight waves deal the
// 256-wide steps of k among themselves and add their sums in LDS, in wave
// order.  In a step a wave reads 16 rows of B by 128 bytes, a lane 32
// consecutive bytes (two blocks) and their two scales, which are neighbouring
// bytes of a word, and the same of A's rows (from the caches), as the matrix
// instructions take them.  Two steps a wave are in flight.
//
// Few columns leave CUs without work: k is then cut into `split` ranges, one
// a workgroup, whose sums a second launch adds in order.
//
// One row by 4096 x 4096: 4.4 us for 8.9 MB, most of it the chain of launch,
// two steps of loads, LDS and store.  (20 x 5120 x 8192: 11.3 us in all, by
// the 64 x 128 tile 18.8.)
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace fp4s {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8, kThreads = 64 * kWaves, kDepth = 2;
static_assert(kFp4SkinnyCols == 16, "one matrix-core tile");

__device__ __forceinline__ i8v wide(i4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// the first n of a chunk's 32 values, the others zero
__device__ __forceinline__ i4 keep(i4 v, int n) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int k = n - 8 * d;
        v[d] = k >= 8 ? v[d] : (k <= 0 ? 0 : (int)((unsigned)v[d] & (0xffffffffu >> (32 - 4 * k))));
    }
    return v;
}

template <int MT>
struct Skinny {
    struct Step {
        i4 b[2], a[MT][2];
        int sb, sa[MT];
    };
    // a row's first byte and its scale words' first byte, at this lane's part of a step
    struct Row {
        const unsigned char *q, *s;
    };
    __device__ __forceinline__ static void load(Step& x, const Row& b, const Row (&a)[MT], const Fp4Args& p, int64_t kt, int lane) {
        const int64_t hb = kt * 2 * p.ldsb * 4, ha = kt * 2 * p.ldsa * 4;
        if (kt * 256 + 256 <= p.K) {
#pragma unroll
            for (int q = 0; q < 2; ++q) x.b[q] = *(const i4*)(b.q + kt * 128 + 16 * q);
            x.sb = *(const unsigned short*)(b.s + hb);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) x.a[i][q] = *(const i4*)(a[i].q + kt * 128 + 16 * q);
                x.sa[i] = *(const unsigned short*)(a[i].s + ha);
            }
            return;
        }
        // the matrix's last step: values past K are zeros in A, and scales past it (which may be NaN) zeros
        const int left = (int)(p.K - kt * 256) - 64 * (lane >> 4);  // values from this lane's first
        const i4 zero = {0, 0, 0, 0};
        const int keep_s = left > 32 ? 0xffff : 0xff;
        x.sb = 0;
        if (left > 0) x.sb = *(const unsigned short*)(b.s + hb) & keep_s;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            x.b[q] = zero;
            if (left > 32 * q) x.b[q] = *(const i4*)(b.q + kt * 128 + 16 * q);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            x.sa[i] = 0;
            if (left > 0) x.sa[i] = *(const unsigned short*)(a[i].s + ha) & keep_s;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                x.a[i][q] = zero;
                if (left > 32 * q) x.a[i][q] = keep(*(const i4*)(a[i].q + kt * 128 + 16 * q), left - 32 * q);
            }
        }
    }
    __device__ __forceinline__ static void multiply(f4 (&acc)[MT], const Step& x) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(x.b[0]), wide(x.a[i][0]), acc[i], 4, 4, 0, x.sb, 0, x.sa[i]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(x.b[1]), wide(x.a[i][1]), acc[i], 4, 4, 1, x.sb, 1, x.sa[i]);
    }

    __device__ __forceinline__ static void run(const Fp4Args& a) {
        __shared__ f4 part[kWaves][MT][64];
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4;
        const int T = a.tiles_m * a.tiles_n;
        const int share = blockIdx.x / T, t = blockIdx.x % T;
        // (row blocks of the same columns side by side)
        const int64_t m0 = (int64_t)(t % a.tiles_m) * (16 * MT), n0 = (int64_t)(t / a.tiles_m) * 16;
        const int64_t steps = (a.K + 255) / 256;
        const int64_t k_lo = share * steps / a.split, k_hi = (share + 1) * steps / a.split;
        // rows past the matrix repeat its last: their results are dropped
        const int64_t n = min<int64_t>(n0 + (lane & 15), a.N - 1);
        const Row rb{a.B + n * a.ldb + 32 * g, (const unsigned char*)(a.sb + (g >> 1) * a.ldsb + n) + 2 * (g & 1)};
        Row ra[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t m = min<int64_t>(m0 + 16 * i + (lane & 15), a.M - 1);
            ra[i] = Row{a.A + m * a.lda + 32 * g, (const unsigned char*)(a.sa + (g >> 1) * a.ldsa + m) + 2 * (g & 1)};
        }
        f4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
        Step x[kDepth];
        int64_t kt = k_lo + wave;
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (kt + d * kWaves < k_hi) load(x[d], rb, ra, a, kt + d * kWaves, lane);
        for (; kt < k_hi; kt += kDepth * kWaves) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (kt + d * kWaves < k_hi) multiply(acc, x[d]);
                if (kt + (d + kDepth) * kWaves < k_hi) load(x[d], rb, ra, a, kt + (d + kDepth) * kWaves, lane);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
        __syncthreads();
        for (int e = tid; e < MT * 256; e += kThreads) {
            const int r = e >> 4, c = e & 15;  // row and column of the tile
            const float* p = (const float*)&part[0][r >> 4][(c >> 2) * 16 + (r & 15)] + (c & 3);
            float v = p[0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += p[w * MT * 256];
            const int64_t m = m0 + r, nn = n0 + c;
            if (m >= a.M || nn >= a.N) continue;
            if (a.split > 1) a.ws[((int64_t)share * a.M + m) * a.N + nn] = v;
            else store_epilogue(a, v, m, nn);
        }
    }
};

template <int MT>
__global__ __launch_bounds__(kThreads) void fp4_skinny_kernel(Fp4Args a) {
    Skinny<MT>::run(a);
}

// the k ranges' sums, in order
__global__ __launch_bounds__(256) void fp4_skinny_sum_kernel(Fp4Args a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, mn = a.M * a.N;
    if (i >= mn) return;
    float v = 0.f;
    for (int s = 0; s < a.split; s += 8) {
        float x[8];  // (in flight together)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s + u < a.split) x[u] = a.ws[(s + u) * mn + i];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s + u < a.split) v += x[u];
    }
    store_epilogue(a, v, i / a.N, i % a.N);
}

}  // namespace fp4s

int launch_fp4_skinny(int rows, const Fp4Args& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n * a.split)), block(fp4s::kThreads);
    if (rows <= 16) hipLaunchKernelGGL(fp4s::fp4_skinny_kernel<1>, grid, block, 0, s, a);
    else if (rows <= 32) hipLaunchKernelGGL(fp4s::fp4_skinny_kernel<2>, grid, block, 0, s, a);
    else if (rows <= 48) hipLaunchKernelGGL(fp4s::fp4_skinny_kernel<3>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(fp4s::fp4_skinny_kernel<4>, grid, block, 0, s, a);
    if (a.split > 1)
        hipLaunchKernelGGL(fp4s::fp4_skinny_sum_kernel, dim3((unsigned)((a.M * a.N + 255) / 256)), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace tcm
