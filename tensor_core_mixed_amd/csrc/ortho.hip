// Newton-Schulz steps that bring a matrix near the nearest orthogonal one,
//
//     X = G / (|G|_F + eps),   X <- a X + (b S + c S^2) X,   S = X X^T,
//
// each singular value s going to a s + b s^3 + c s^5 and the singular vectors
// staying (X is G or, where G has more rows than columns, its transpose).
//
// Every matrix is held in two binary16 parts, value * 2^e = upper + lower: 22
// bits, of which products keep all but lower times lower (2^-22).  Over five
// steps that is as exact as binary32 throughout (2.0e-6 against 3.0e-6 of a
// 768 x 2048 update, from 64 bits; one binary16 part would give 1.4e-3, two
// bfloat16 ones 2.6e-5), in three matrix instructions of sixteen times binary32's
// rate.  The exponents e come from bounds: singular values of X lie below 1
// at first, then below the largest |a s + b s^3 + c s^5| there, and entries
// below singular values; so nothing passes binary16's range whatever G and
// the coefficients are.
//
// One exponent a matrix costs bits where its parts differ in size: lower parts
// end at 2^-24, so a value is held to 2^-38 of the bound at best, and those
// below 2^-39 are zeros.  Rows of 2^-p of the others', brought to 1 by steps
// (1.5, -0.5, 0), are off by 5e-7 of themselves at p = 12, 8e-6 at 16, 1.4e-4
// at 20 and 2e-3 at 24, where binary32 stays at 2e-7; five of Muon's steps of
// such a matrix at p = 20 are off by 1.7e-6 of the whole.  (Three bfloat16
// parts have binary32's range and bits, in six instructions.)
//
// Parts lie as the main loop of pair_tile.h takes them: rows of 128-byte
// pieces, 32 upper parts then their 32 lower ones; rows end in zeros up to a
// piece.  X is held as it is and transposed, since the first product runs
// along its rows and the last along its columns:
//
//     S = X X^T and T = b S + c S S (S is symmetric) only where tile row >=
//         tile column; the others are those transposed,
//     X = a X + T X, with rows of X transposed as second operand; its
//         tiles leave as they are and transposed (through LDS, a wave its own
//         64 x 32 values at a time) for the next step.  (a within T, on the
//         diagonal, would save reading X here and lose bits of a X.)
//
// Few tiles leave CUs without work: k is cut into two halves within a
// workgroup of the smallest tiles (their sum goes through LDS) and into
// ranges, one a workgroup, and a second launch adds the partial tiles in order
// and finishes them.
//
// Five steps of 4096 x 1024 take 345 to 364 us: 209 GFLOP of binary16, 144 us
// at the rate that a library product of 8192^3 reaches (1458 TFLOP/s), the
// rest being the launches' fill, the way out of 48 MB of X a step and copies
// that arrive late (matrix cores busy in 48 and 45% of S's and X's cycles, in
// 23% of T's, which has 136 workgroups of four waves).  Eight 768 x 2048: 665 to 690 us
// (floor 336), 4096 x 4096: 3640 (2830).  128 x 128 tiles are taken by eight waves with copies two steps
// ahead (S of 4096 x 1024 19 us and X 31; by two groups of four waves, one
// step ahead, 21 and 36), 64 x 64 by two groups, two steps ahead (512 x 512
// 154 us in all; by four groups, one step ahead, 170).  Shorter sides up to
// 128: ortho_small.hip.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"
#include "ortho_util.h"
#include "pair_tile.h"

namespace tcm {
namespace ortho {

using pair::f4;
typedef unsigned u4_t __attribute__((ext_vector_type(4)));

// N consecutive values' parts (N a multiple of 8) at column c, a multiple of N, of the row at p
template <int N>
__device__ __forceinline__ void store_parts(char* row, int64_t c, const unsigned (&w)[N]) {
    char* p = row + (c >> 5) * 128 + (c & 31) * 2;
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        u4_t hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = upper2(w[8 * q + 2 * i], w[8 * q + 2 * i + 1]), lo[i] = lower2(w[8 * q + 2 * i], w[8 * q + 2 * i + 1]);
        *(u4_t*)(p + 16 * q) = hi;
        *(u4_t*)(p + 64 + 16 * q) = lo;
    }
}
// 16 consecutive values of the row at p
__device__ __forceinline__ void load_parts(float (&v)[16], const char* row, int64_t c) {
    const char* p = row + (c >> 5) * 128 + (c & 31) * 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const u4_t hi = *(const u4_t*)(p + 16 * q), lo = *(const u4_t*)(p + 64 + 16 * q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned a = hi[i >> 1], b = lo[i >> 1];  // (a bit_cast of a vector's element takes its first)
            const h2_t x = __builtin_bit_cast(h2_t, a), y = __builtin_bit_cast(h2_t, b);
            v[8 * q + i] = (float)x[i & 1] + (float)y[i & 1];
        }
    }
}
// n of N consecutive values in O's type to any address
template <int N>
__device__ __forceinline__ void store_out(char* p, const float (&v)[N], int type, int64_t n) {
    if (n >= N) {
        if (type == C_ACC) {
            __builtin_memcpy(p, v, 4 * N);
        } else {
            unsigned w[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const unsigned lo = type == C_F16 ? __builtin_bit_cast(unsigned short, (_Float16)v[2 * i]) : __builtin_bit_cast(unsigned short, (__bf16)v[2 * i]);
                const unsigned hi = type == C_F16 ? __builtin_bit_cast(unsigned short, (_Float16)v[2 * i + 1]) : __builtin_bit_cast(unsigned short, (__bf16)v[2 * i + 1]);
                w[i] = lo | hi << 16;
            }
            __builtin_memcpy(p, w, 2 * N);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) store_c_any(p + i * c_elem_bytes(type), type, v[i]);
    }
}

// ---- G's norm, and X's parts

constexpr int kThreads = 256;

// the sum of squares of a slice of an entry of G, in binary64: no binary32 value passes its range
template <int XT>
__global__ __launch_bounds__(kThreads) void norm_kernel(OrthoArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2, N = 8;
    __shared__ double part[kThreads / 64];
    const int64_t entry = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
    const char* g = (const char*)a.g + entry * a.stride_g * ES;
    const unsigned per_row = (unsigned)((a.cols + N - 1) / N);
    double s = 0;
    // pieces of N values, in a row's order: this thread's first, and how far it goes on
    const int64_t first = slice * kThreads + threadIdx.x, hop = a.slices * kThreads;
    int64_t r = first / per_row, c = first % per_row;
    const int64_t hop_r = hop / per_row, hop_c = hop % per_row;
#pragma unroll 2
    for (; r < a.rows; r += hop_r, c += hop_c) {
        if (c >= per_row) c -= per_row, ++r;
        if (r >= a.rows) break;
        const char* p = g + (r * a.ldg + c * N) * ES;
        if (c * N + N <= a.cols) {
            unsigned w[N * ES / 4];
            __builtin_memcpy(w, p, N * ES);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const double v = (double)load_float<XT>((const char*)w, j);
                s = __builtin_fma(v, v, s);
            }
        } else {
            for (int64_t j = 0; c * N + j < a.cols; ++j) {
                const double v = (double)load_float<XT>(p, j);
                s = __builtin_fma(v, v, s);
            }
        }
    }
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.squares[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// G times its inverse norm and `factor`: its parts, as it lies and transposed (64 x 64 values a workgroup), or with
// OUT rounded to O
template <int XT, bool OUT>
__global__ __launch_bounds__(kThreads) void start_kernel(OrthoArgs a, float factor) {
    constexpr int ES = XT == F32 ? 4 : 2;
    __shared__ unsigned tr[64 * 65];
    const int64_t tc = (a.cols_pad + 63) / 64, tiles = tc * ((a.rows_pad + 63) / 64);
    const int64_t b = a.first_tile + blockIdx.x, entry = b / tiles, t = b % tiles;
    const int64_t r0 = t / tc * 64, c0 = t % tc * 64;
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
    const char* g = (const char*)a.g + (entry * a.stride_g + (r0 + r) * a.ldg + c0 + c) * ES;
    float v[16];
    const int64_t n = r0 + r < a.rows ? a.cols - c0 - c : 0;
    if (n >= 16) {
        unsigned w[4 * ES];
        __builtin_memcpy(w, g, 16 * ES);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = load_float<XT>((const char*)w, j);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = j < n ? load_float<XT>(g, j) : 0.f;
    }
    const double f = inverse_norm(a, entry) * (double)factor;
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = j < n ? (float)((double)v[j] * f) : 0.f;  // (zeros past the matrix, also under a NaN norm)
    if constexpr (OUT) {
        if (n > 0) store_out((char*)a.o + (entry * a.stride_o + (r0 + r) * a.ldo + c0 + c) * c_elem_bytes(a.o_type), v, a.o_type, n);
    } else {
        unsigned w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) tr[(c + j) * 65 + r] = w[j] = split(v[j]);
        if (r0 + r < a.rows && c0 + c < a.cols_pad) store_parts(a.as_is + entry * a.entry_bytes + (r0 + r) * a.cols_pad * 4, c0 + c, w);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = tr[r * 65 + c + j];
        if (c0 + r < a.cols && r0 + c < a.rows_pad) store_parts(a.across + entry * a.entry_bytes + (c0 + r) * a.rows_pad * 4, r0 + c, w);
    }
}

// ---- the products

template <int CFG>
struct Tile {
    using L = pair::Loop<kOrthoTiles[CFG].bm, kOrthoTiles[CFG].bn, kOrthoTiles[CFG].wm, kOrthoTiles[CFG].wn, kOrthoTiles[CFG].stages, false,
                         false>;
    static constexpr int FM = L::FM, PARTS = kOrthoTiles[CFG].parts, NT = L::NT * PARTS, LDS = L::LDS * PARTS;
    static_assert(FM % 2 == 0, "a wave's rows in pairs of tiles");
    static constexpr int kPitch = 33, kWaveWords = 64 * kPitch;

    // Tile t of an entry's: all of them, or those on and under the diagonal.
    __device__ __forceinline__ static void tile_at(const OrthoMul& p, int t, int* tm, int* tn) {
        if (p.symmetric) {
            int i = (int)((__builtin_sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
            while (i * (i + 1) / 2 > t) --i;
            while ((i + 1) * (i + 2) / 2 <= t) ++i;
            *tm = i;
            *tn = t - i * (i + 1) / 2;
        } else {
            super_order(t, p.tiles_m, p.tiles_n, p.group_m, p.super_m, p.super_n, tm, tn);
        }
    }

    // 32 rows from m0 by 64 columns from n0 of an entry: v = alpha * acc + beta * P, to D and transposed to E.
    __device__ __forceinline__ static void finish(const f4 (&acc)[2][4], const OrthoMul& p, int64_t entry, int64_t m0, int64_t n0, bool across,
                                                  unsigned* lds, int lane) {
        const int64_t n = n0 + 16 * (lane >> 4);
        float v[2][16];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t m = m0 + 16 * u + (lane & 15);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[u][e] = p.alpha * acc[u][e >> 2][e & 3];
            if (p.P && m < p.M && n < p.n_pad) {
                float x[16];
                load_parts(x, p.P + entry * p.entry_bytes + m * p.n_pad * 4, n);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[u][e] = __builtin_fmaf(p.beta, x[e], v[u][e]);
            }
        }
        if (p.out) {
            const int es = c_elem_bytes(p.out_type);
            char* o = p.out + entry * p.stride_out * es;
            if (!p.out_across) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int64_t m = m0 + 16 * u + (lane & 15);
                    if (m < p.M && n < p.N) store_out(o + (m * p.ld_out + n) * es, v[u], p.out_type, p.N - n);
                }
                return;
            }
            float* f = (float*)lds;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) f[(16 * (lane >> 4) + e) * kPitch + 16 * u + (lane & 15)] = v[u][e];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 16 * q + (lane >> 2), c = 8 * (lane & 3);
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = f[r * kPitch + c + i];
                if (n0 + r < p.N && m0 + c < p.M) store_out(o + ((n0 + r) * p.ld_out + m0 + c) * es, w, p.out_type, p.M - m0 - c);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            return;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t m = m0 + 16 * u + (lane & 15);
            unsigned w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = split(v[u][e]);
            if (m < p.M && n < p.n_pad) store_parts(p.D + entry * p.entry_bytes + m * p.n_pad * 4, n, w);
            if (across) {
#pragma unroll
                for (int e = 0; e < 16; ++e) lds[(16 * (lane >> 4) + e) * kPitch + 16 * u + (lane & 15)] = w[e];
            }
        }
        if (!across) return;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 16 * q + (lane >> 2), c = 8 * (lane & 3);
            unsigned w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = lds[r * kPitch + c + i];
            if (n0 + r < p.N && m0 + c < p.m_pad) store_parts(p.E + entry * p.entry_bytes + (n0 + r) * p.m_pad * 4, m0 + c, w);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }

    __device__ __forceinline__ static void run(const OrthoMul& p) {
        __shared__ __attribute__((aligned(1024))) char smem_raw[LDS];
        constexpr int kSums = (PARTS - 1) * L::NT * FM * 16;  // words of the other parts' sums
        static_assert((kSums + L::NW * kWaveWords) * 4 <= LDS, "");
        const int tid = threadIdx.x, lane = tid & 63;
        const int id = __builtin_amdgcn_readfirstlane(tid >> 6), part = id / L::NW, wave = id % L::NW;
        const int wm = wave / L::WN, wn = wave % L::WN;
        const int nidx = xcd_order(blockIdx.x, p.tiles * p.split * p.batch);
        const int entry = nidx / (p.tiles * p.split), rest = nidx - entry * p.tiles * p.split;
        const int share = rest / p.tiles, t = rest - share * p.tiles;
        int tm, tn;
        tile_at(p, t, &tm, &tn);
        const int64_t m0 = (int64_t)tm * L::BM, n0 = (int64_t)tn * L::BN;
        const int64_t steps = p.k_pad / 32;
        const int lo = (int)(share * steps / p.split), hi = (int)((share + 1) * steps / p.split);
        const int each = (hi - lo + PARTS - 1) / PARTS, k_lo = lo + part * each, k_hi = min(k_lo + each, hi);
        f4 acc[FM][4];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
        const pair::Operands o{(const unsigned char*)p.A + entry * p.entry_bytes, (const unsigned char*)p.B + entry * p.entry_bytes, p.M, p.N,
                               p.k_pad * 4, p.k_pad * 4, p.k_pad * 4, 0, nullptr, nullptr, 0, 0};
        L::run(acc, o, (pair::lds_char*)smem_raw + part * L::LDS, m0, n0, k_lo, k_hi, each, wave, lane);
        __syncthreads();  // (every wave is done with the operands in LDS)
        if constexpr (PARTS > 1) {
            // the first part adds the others' sums, in order, and finishes the tile
            f4* lds = (f4*)smem_raw;
            if (part) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) lds[((id - L::NW) * FM * 4 + i * 4 + j) * 64 + lane] = acc[i][j];
            }
            __syncthreads();
            if (part) return;
#pragma unroll
            for (int q = 0; q < PARTS - 1; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] += lds[((q * L::NW + wave) * FM * 4 + i * 4 + j) * 64 + lane];
        }
        if (p.split > 1) {
            f4* w = (f4*)p.ws + ((int64_t)nidx * L::NW + wave) * FM * 4 * 64 + lane;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[(i * 4 + j) * 64] = acc[i][j];
            return;
        }
        const bool across = p.E && !(p.symmetric && tm == tn);
#pragma unroll
        for (int i = 0; i < FM; i += 2) {
            f4 two[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) two[0][j] = acc[i][j], two[1][j] = acc[i + 1][j];
            finish(two, p, entry, m0 + wm * L::TM + 16 * i, n0 + wn * 64, across, (unsigned*)smem_raw + kSums + wave * kWaveWords, lane);
        }
    }

    // The sum of a split launch: four waves take two row tiles of one of its waves, each adds the ranges of two of the
    // eight accumulators (many of their reads in flight), and one finishes them.
    __device__ __forceinline__ static void run_sum(const OrthoMul& p) {
        __shared__ __attribute__((aligned(16))) unsigned lds[kWaveWords];
        const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
        int64_t b = blockIdx.x;
        const int i = (int)(b % (FM / 2)) * 2;
        b /= FM / 2;
        const int wave = (int)(b % L::NW);
        b /= L::NW;
        const int t = (int)(b % p.tiles);
        const int64_t entry = b / p.tiles;
        int tm, tn;
        tile_at(p, t, &tm, &tn);
        const int wm = wave / L::WN, wn = wave % L::WN;
        const f4* w = (const f4*)p.ws + (((entry * p.split * p.tiles + t) * L::NW + wave) * FM + i) * 4 * 64 + 2 * q * 64 + lane;
        const int64_t step = (int64_t)p.tiles * L::NW * FM * 4 * 64;
        f4 s[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
        for (int k = 0; k < p.split; k += 8) {
            f4 x[8][2];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < p.split) x[u][0] = w[(k + u) * step], x[u][1] = w[(k + u) * step + 64];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < p.split) s[0] += x[u][0], s[1] += x[u][1];
        }
        f4* l = (f4*)lds;
        l[(2 * q) * 64 + lane] = s[0];
        l[(2 * q + 1) * 64 + lane] = s[1];
        __syncthreads();
        if (q) return;
        f4 two[2][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) two[j >> 2][j & 3] = l[j * 64 + lane];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (before finish() writes there)
        finish(two, p, entry, (int64_t)tm * L::BM + wm * L::TM + 16 * i, (int64_t)tn * L::BN + wn * 64, p.E && !(p.symmetric && tm == tn), lds, lane);
    }
};

template <int CFG>
__global__ __launch_bounds__((Tile<CFG>::NT)) __attribute__((amdgpu_waves_per_eu(2))) void ortho_tile_kernel(OrthoMul p) {
    Tile<CFG>::run(p);
}
template <int CFG>
__global__ __launch_bounds__(256) void ortho_sum_kernel(OrthoMul p) {
    Tile<CFG>::run_sum(p);
}

template <int CFG>
int launch_mul(const OrthoMul& p, hipStream_t s) {
    using X = Tile<CFG>;
    const int64_t tiles = (int64_t)p.tiles * p.batch;
    hipLaunchKernelGGL(ortho_tile_kernel<CFG>, dim3((unsigned)(tiles * p.split)), dim3(X::NT), 0, s, p);
    if (p.split > 1) hipLaunchKernelGGL(ortho_sum_kernel<CFG>, dim3((unsigned)(tiles * X::L::NW * X::FM / 2)), dim3(256), 0, s, p);
    return (int)hipGetLastError();
}

template <int XT>
int launch_norm(const OrthoArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(norm_kernel<XT>, dim3((unsigned)(a.batch * a.slices)), dim3(kThreads), 0, s, a);
    return (int)hipGetLastError();
}
template <int XT>
int launch_start(const OrthoArgs& a, float factor, bool out, hipStream_t s) {
    const int64_t tiles = a.batch * ((a.cols_pad + 63) / 64) * ((a.rows_pad + 63) / 64), most = (int64_t)1 << 23;  // (threads: 32 bits)
    for (int64_t t = 0; t < tiles; t += most) {
        OrthoArgs e = a;
        e.first_tile = t;
        const dim3 grid((unsigned)(tiles - t < most ? tiles - t : most));
        if (out) hipLaunchKernelGGL((start_kernel<XT, true>), grid, dim3(kThreads), 0, s, e, factor);
        else hipLaunchKernelGGL((start_kernel<XT, false>), grid, dim3(kThreads), 0, s, e, factor);
    }
    return (int)hipGetLastError();
}

}  // namespace ortho

int launch_ortho_norm(int x_type, const OrthoArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return ortho::launch_norm<F16>(a, s);
    case BF16: return ortho::launch_norm<BF16>(a, s);
    default: return ortho::launch_norm<F32>(a, s);
    }
}
int launch_ortho_start(int x_type, const OrthoArgs& a, float factor, bool out, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return ortho::launch_start<F16>(a, factor, out, s);
    case BF16: return ortho::launch_start<BF16>(a, factor, out, s);
    default: return ortho::launch_start<F32>(a, factor, out, s);
    }
}
int launch_ortho_mul(int cfg, const OrthoMul& p, void* stream) {
    static_assert(kNumOrthoTiles == 3, "one case a config");
    hipStream_t s = (hipStream_t)stream;
    return cfg == 0 ? ortho::launch_mul<0>(p, s) : (cfg == 1 ? ortho::launch_mul<1>(p, s) : ortho::launch_mul<2>(p, s));
}

}  // namespace tcm
