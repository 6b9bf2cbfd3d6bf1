// Block-scaled 8-bit product of a few rows (a decoding batch): B is read once
// and binds the time, so its bytes go straight from memory to registers.
//
// A workgroup takes 16 columns and up to 64 rows; its eight waves deal the
// 128-wide k blocks among themselves and add their sums in LDS, in wave
// order.  A wave reads 16 rows of B by 128 bytes (32 bytes a lane) and the
// same k of A's rows (from the caches), takes both to 16-bit floats, which
// hold them exactly, and multiplies on 16x16x32 MFMAs; the blocks' sums are
// scaled and added in binary32.  One block a wave is in flight: the waves of
// two or more workgroups a CU cover the rest (with two or four blocks a wave
// 16 rows of 4096 x 4096 took 7.3 and 7.7 us, with one 7.1; 37 of 5120 x 8192
// 33 and 30).  One row of 8192 x 8192 takes 16.7 us, 4.0 TB/s; more rows cost
// their reads of A, every workgroup all of it.
//
// Few columns leave CUs without work: k is then cut into `split` ranges, one
// a workgroup, whose sums a second launch adds in order.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace fp8s {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
static_assert(kFp8SkinnyCols == 16, "one matrix-core tile");

// 16 bytes of a row from k on, zeros from K on.  (A chunk with a byte before
// K is read whole: rows lie at multiples of 16 bytes, so it ends within the
// page of that byte.)
__device__ __forceinline__ i4 load16(const unsigned char* p, int64_t k, int64_t K) {
    i4 v = {0, 0, 0, 0};
    if (k < K) v = *(const i4*)(p + k);
    const int n = (int)(K - k < 16 ? K - k : 16);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int r = n - 4 * d;
        v[d] = r >= 4 ? v[d] : (r <= 0 ? 0 : (int)((unsigned)v[d] & (0xffffffffu >> (32 - 8 * r))));
    }
    return v;
}

template <bool A5, bool B5, bool BROW, int MT>
struct Skinny {
    struct Block {
        i4 b[2], a[MT][2];
        float sa[MT];
        f4 sb;
    };
    struct Src {
        const unsigned char *b, *a[MT];
        const float *sa[MT], *sb;
        int cols;  // of sb's four columns the last that exists
    };
    __device__ __forceinline__ static void load(Block& x, const Src& s, const Fp8Args& a, int64_t kt, int lane) {
        const int64_t k = kt * 128 + 16 * (lane >> 4);  // (four lanes read 64 consecutive bytes)
        if (kt * 128 + 128 <= a.K) {
#pragma unroll
            for (int q = 0; q < 2; ++q) x.b[q] = *(const i4*)(s.b + k + 64 * q);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) x.a[i][q] = *(const i4*)(s.a[i] + k + 64 * q);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) x.b[q] = load16(s.b, k + 64 * q, a.K);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) x.a[i][q] = load16(s.a[i], k + 64 * q, a.K);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) x.sa[i] = s.sa[i][kt * a.ldsa];
        if constexpr (BROW) {
#pragma unroll
            for (int r = 0; r < 4; ++r) x.sb[r] = s.sb[kt * a.ldsb + min(r, s.cols)];
        } else {
            x.sb[0] = s.sb[kt];
        }
    }
    __device__ __forceinline__ static void multiply(f4 (&acc)[MT], const Block& x) {
        f16x8_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = fp8_to_f16x8<B5>(x.b[q >> 1][2 * (q & 1)], x.b[q >> 1][2 * (q & 1) + 1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            f4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                p = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    b[q], fp8_to_f16x8<A5>(x.a[i][q >> 1][2 * (q & 1)], x.a[i][q >> 1][2 * (q & 1) + 1]), p, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(p[r], x.sa[i] * x.sb[BROW ? r : 0], acc[i][r]);
        }
    }

    __device__ __forceinline__ static void run(const Fp8Args& a) {
        __shared__ f4 part[kWaves][MT][64];
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int T = a.tiles_m * a.tiles_n;
        const int share = blockIdx.x / T, t = blockIdx.x % T;
        // (row blocks of the same columns side by side)
        const int64_t m0 = (int64_t)(t % a.tiles_m) * (16 * MT), n0 = (int64_t)(t / a.tiles_m) * 16;
        const int64_t steps = scale_blocks(a.K);
        const int64_t k_lo = share * steps / a.split, k_hi = (share + 1) * steps / a.split;
        // rows past the matrix repeat its last: their results are dropped
        Src s;
        const int64_t n = min<int64_t>(n0 + (lane & 15), a.N - 1);
        s.b = a.B + n * a.ldb;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t m = min<int64_t>(m0 + 16 * i + (lane & 15), a.M - 1);
            s.a[i] = a.A + m * a.lda;
            s.sa[i] = a.sa + m;
        }
        const int64_t nb = min<int64_t>(n0 + 4 * (lane >> 4), a.N - 1);
        s.cols = (int)min<int64_t>(3, a.N - 1 - nb);
        s.sb = BROW ? a.sb + nb : a.sb + n0 / kScaleBlock * a.ldsb;
        f4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
        Block x;
        int64_t kt = k_lo + wave;
        if (kt < k_hi) load(x, s, a, kt, lane);
        for (; kt < k_hi; kt += kWaves) {
            multiply(acc, x);
            if (kt + kWaves < k_hi) load(x, s, a, kt + kWaves, lane);
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

template <bool A5, bool B5, bool BROW, int MT>
__global__ __launch_bounds__(kThreads) void fp8_skinny_kernel(Fp8Args a) {
    Skinny<A5, B5, BROW, MT>::run(a);
}

// the k ranges' sums, in order
__global__ __launch_bounds__(256) void fp8_skinny_sum_kernel(Fp8Args a) {
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

template <bool A5, bool B5, bool BROW>
void launch_rows(const Fp8Args& a, int rows, hipStream_t s) {
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n * a.split)), block(kThreads);
    if (rows <= 16) hipLaunchKernelGGL((fp8_skinny_kernel<A5, B5, BROW, 1>), grid, block, 0, s, a);
    else if (rows <= 32) hipLaunchKernelGGL((fp8_skinny_kernel<A5, B5, BROW, 2>), grid, block, 0, s, a);
    else if (rows <= 48) hipLaunchKernelGGL((fp8_skinny_kernel<A5, B5, BROW, 3>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((fp8_skinny_kernel<A5, B5, BROW, 4>), grid, block, 0, s, a);
}
template <bool A5, bool B5>
void launch_scales(const Fp8Args& a, int rows, hipStream_t s) {
    if (a.b_row) launch_rows<A5, B5, true>(a, rows, s);
    else launch_rows<A5, B5, false>(a, rows, s);
}

}  // namespace fp8s

int launch_fp8_skinny(int rows, const Fp8Args& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (a.a_e5m2) {
        if (a.b_e5m2) fp8s::launch_scales<true, true>(a, rows, s);
        else fp8s::launch_scales<true, false>(a, rows, s);
    } else {
        if (a.b_e5m2) fp8s::launch_scales<false, true>(a, rows, s);
        else fp8s::launch_scales<false, false>(a, rows, s);
    }
    if (a.split > 1)
        hipLaunchKernelGGL(fp8s::fp8_skinny_sum_kernel, dim3((unsigned)((a.M * a.N + 255) / 256)), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace tcm
