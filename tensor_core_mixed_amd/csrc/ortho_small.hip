// Newton-Schulz steps of matrices whose shorter side is at most 128: the
// formulas and two-part binary16 values of ortho.hip, with few launches.
//
// A workgroup owns a chunk of an entry's columns of X (CW of them, all NP
// rows), held in LDS transposed, and as it lies while S is summed from it:
//
//     S = X X^T          over the chunk's columns,
//     T = b S + c S S    in every workgroup of the entry anew (n^3 is little),
//     X = a X + T X      on the chunk alone.
//
// So a step needs one thing from elsewhere, the other chunks' share of S.  An
// entry of one chunk runs all its steps in one launch, with its norm; others
// take a launch a step, which starts with the sum of all chunks' shares in
// order, after one that scales X.  T and X as it lies share their place in
// LDS: they are never needed at once.
//
// Five steps of 64 x 64 take 32 us (80 in the 17 launches of ortho.hip), of
// 128 x 128 59 (100), a thousand of them 126 and 237 (320 and 787); 16 of
// 64 x 4096 113 (197).  A step of one chunk is 4.2 us at 64 rows and 9.7 at
// 128, where the products alone are 3.9: the rest are the ways through LDS
// between the three of them and their barriers.  Tried without gain: the
// k loop unrolled, products of one accumulator in a row.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"
#include "ortho_util.h"

namespace tcm {
namespace ortho {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef unsigned u2_t __attribute__((ext_vector_type(2)));
typedef unsigned u4_t __attribute__((ext_vector_type(4)));

template <int NP>
struct Small {
    static constexpr int NT = 512, NW = 8, CW = kOrthoSmallElems / NP;
    // Rows in LDS: upper parts, lower parts, and 16 bytes that spread the rows over the banks.
    static constexpr int XT_PITCH = NP * 4 + 16, XT_LOW = NP * 2;  // X transposed [CW][NP], and S and T [NP][NP]
    static constexpr int X_PITCH = CW * 4 + 16, X_LOW = CW * 2;    // X [NP][CW]
    static constexpr int XT_BYTES = CW * XT_PITCH, X_BYTES = NP * X_PITCH, S_BYTES = NP * XT_PITCH;
    static constexpr int LDS = XT_BYTES + (X_BYTES > S_BYTES ? X_BYTES : S_BYTES);
    static_assert(LDS <= 159 * 1024, "");
    // Tiles of 16 x 16: of S and T a wave takes SR x 2, of X 4 x 2.
    static constexpr int SR = NP == 64 ? 1 : 4;
    static_assert((NP == 64 || NP == 128) && NW * 2 * SR * 256 == NP * NP && NW * 8 * 256 == NP * CW, "");

    __device__ __forceinline__ static h8 frag(const char* p) { return *(const h8*)p; }
    // acc[r][c] += rows a + 16 r of one matrix by rows b + 16 c of another, `steps` pieces of 32 k: all products of two
    // parts but lower times lower
    template <int R>
    __device__ __forceinline__ static void multiply(f4 (&acc)[R][2], const char* a, int a_pitch, int a_low, const char* b, int b_pitch, int b_low,
                                                    int steps) {
        const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
        a += i * a_pitch + g * 16;
        b += i * b_pitch + g * 16;
        for (int k = 0; k < steps; ++k) {
            h8 af[R][2], bf[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int q = 0; q < 2; ++q) bf[c][q] = frag(b + 64 * k + 16 * c * b_pitch + q * b_low);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q < 2; ++q) af[r][q] = frag(a + 64 * k + 16 * r * a_pitch + q * a_low);
#pragma unroll
            for (int q = 0; q < 3; ++q)  // (one product of every accumulator after another: each waits for its last)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[r][q == 2], bf[c][q == 1], acc[r][c], 0, 0, 0);
        }
    }
    // four values at columns c .. c + 3 (c a multiple of 4) of the row at p
    __device__ __forceinline__ static void store4(char* p, int low, int c, const unsigned (&w)[4]) {
        *(u2_t*)(p + 2 * c) = u2_t{upper2(w[0], w[1]), upper2(w[2], w[3])};
        *(u2_t*)(p + low + 2 * c) = u2_t{lower2(w[0], w[1]), lower2(w[2], w[3])};
    }
    __device__ __forceinline__ static void load4(float (&v)[4], const char* p, int low, int c) {
        const u2_t hi = *(const u2_t*)(p + 2 * c), lo = *(const u2_t*)(p + low + 2 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned a = hi[e >> 1], b = lo[e >> 1];  // (a bit_cast of a vector's element takes its first)
            const h2_t x = __builtin_bit_cast(h2_t, a), y = __builtin_bit_cast(h2_t, b);
            v[e] = (float)x[e & 1] + (float)y[e & 1];
        }
    }
    __device__ __forceinline__ static void store1(char* p, int low, int c, unsigned w) {
        *(unsigned short*)(p + 2 * c) = (unsigned short)w;
        *(unsigned short*)(p + low + 2 * c) = (unsigned short)(w >> 16);
    }

    template <int XT>
    __device__ __forceinline__ static void run(const OrthoSmallArgs& p) {
        constexpr int ES = XT == F32 ? 4 : 2, PER = NP * CW / NT;
        __shared__ __attribute__((aligned(16))) char lds[LDS];
        __shared__ double part[NW];
        char *xt = lds, *rg = lds + XT_BYTES;  // rg: X as it lies, or S or T
        const OrthoArgs& a = p.g;
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
        const int64_t entry = blockIdx.x / p.chunks;
        const int chunk = (int)(blockIdx.x % p.chunks);
        const int64_t col0 = (int64_t)chunk * CW;
        const int cols = (int)(p.m - col0 < CW ? p.m - col0 : CW);
        const int k_n = (p.n + 31) / 32, k_m = (cols + 31) / 32;
        const int s_row = NP == 64 ? (wave >> 1) * 16 : (wave & 1) * 64, s_col = NP == 64 ? (wave & 1) * 32 : (wave >> 1) * 32;
        const int x_row = NP == 64 ? 0 : (wave & 1) * 64, x_col = NP == 64 ? wave * 32 : (wave >> 1) * 32;
        f4* share = (f4*)p.shares_out + (entry * p.chunks + chunk) * (NP * NP / 4);
        char* state = p.state + (entry * p.chunks + chunk) * (int64_t)(NP * CW * 4);

        f4 s[SR][2];
        const auto sum_s = [&] {  // the chunk's share of S, from rg
#pragma unroll
            for (int r = 0; r < SR; ++r) s[r][0] = s[r][1] = f4{0.f, 0.f, 0.f, 0.f};
            multiply<SR>(s, rg + s_row * X_PITCH, X_PITCH, X_LOW, rg + s_col * X_PITCH, X_PITCH, X_LOW, k_m);
        };
        const auto keep = [&] {  // X and S's share for the next launch
            for (int q = tid; q < NP * CW / 4; q += NT) {
                const int c = q / (NP / 4), o = q % (NP / 4) * 16;
                ((u4_t*)state)[q] = *(const u4_t*)(xt + c * XT_PITCH + o);
            }
#pragma unroll
            for (int r = 0; r < SR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) share[((wave * SR + r) * 2 + c) * 64 + lane] = s[r][c];
        };
        if (p.first) {
            const char* x = (const char*)a.g + (entry * a.stride_g + col0 * (p.tall ? a.ldg : 1)) * ES;
            float v[PER];
#pragma unroll
            for (int q = 0; q < PER; ++q) {  // (a wave's lanes run along G's rows)
                const int e = q * NT + tid, n = p.tall ? e % NP : e / CW, c = p.tall ? e / NP : e % CW;
                const bool in = n < p.n && c < cols;
                v[q] = load_float<XT>(x, in ? (p.tall ? c * a.ldg + n : n * a.ldg + c) : 0);  // (no branch: all loads in flight)
                v[q] = in ? v[q] : 0.f;
            }
            double inverse;
            if (a.squares) {
                inverse = inverse_norm(a, entry);
            } else {  // (all of G is here)
                double sq = 0;
#pragma unroll
                for (int q = 0; q < PER; ++q) sq = __builtin_fma((double)v[q], (double)v[q], sq);
                for (int o = 32; o; o >>= 1) sq += __shfl_xor(sq, o);
                if (lane == 0) part[wave] = sq;
                __syncthreads();
                sq = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) sq += part[w];
                inverse = 1 / (sqrt(sq) + (double)a.eps);
            }
            const double f = inverse * (double)p.factor;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int e = q * NT + tid, n = p.tall ? e % NP : e / CW, c = p.tall ? e / NP : e % CW;
                // (zeros past the matrix, also under a NaN norm)
                const unsigned w = n < p.n && c < cols ? split((float)((double)v[q] * f)) : 0u;
                store1(xt + c * XT_PITCH, XT_LOW, n, w);
                store1(rg + n * X_PITCH, X_LOW, c, w);
            }
            __syncthreads();
            sum_s();
        } else {
            for (int q = tid; q < NP * CW / 4; q += NT) {
                const int c = q / (NP / 4), o = q % (NP / 4) * 16;
                *(u4_t*)(xt + c * XT_PITCH + o) = ((const u4_t*)state)[q];
            }
#pragma unroll
            for (int r = 0; r < SR; ++r) s[r][0] = s[r][1] = f4{0.f, 0.f, 0.f, 0.f};
            const f4* from = (const f4*)p.shares_in + entry * p.chunks * (NP * NP / 4) + wave * SR * 2 * 64 + lane;
            for (int q = 0; q < p.chunks; q += 4) {
                f4 w[4][SR][2];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int r = 0; r < SR; ++r)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (q + u < p.chunks) w[u][r][c] = from[(q + u) * (NP * NP / 4) + (r * 2 + c) * 64];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int r = 0; r < SR; ++r)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (q + u < p.chunks) s[r][c] += w[u][r][c];
            }
        }
        for (int k = 0; k < p.steps; ++k) {
            const OrthoStep& f = p.step[k];
            __syncthreads();  // (X as it lies has been read)
#pragma unroll
            for (int r = 0; r < SR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    unsigned w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][c][e] *= f.s_alpha, w[e] = split(s[r][c][e]);
                    store4(rg + (s_col + 16 * c + i) * XT_PITCH, XT_LOW, s_row + 16 * r + 4 * g, w);  // (S is symmetric)
                }
            __syncthreads();
            f4 t[SR][2];
#pragma unroll
            for (int r = 0; r < SR; ++r) t[r][0] = t[r][1] = f4{0.f, 0.f, 0.f, 0.f};
            multiply<SR>(t, rg + s_row * XT_PITCH, XT_PITCH, XT_LOW, rg + s_col * XT_PITCH, XT_PITCH, XT_LOW, k_n);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < SR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    unsigned w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = split(__builtin_fmaf(f.t_beta, s[r][c][e], f.t_alpha * t[r][c][e]));
                    store4(rg + (s_col + 16 * c + i) * XT_PITCH, XT_LOW, s_row + 16 * r + 4 * g, w);
                }
            __syncthreads();
            f4 x[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r][0] = x[r][1] = f4{0.f, 0.f, 0.f, 0.f};
            if (x_col < cols)
                multiply<4>(x, rg + x_row * XT_PITCH, XT_PITCH, XT_LOW, xt + x_col * XT_PITCH, XT_PITCH, XT_LOW, k_n);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float old[4];
                    load4(old, xt + (x_col + 16 * c + i) * XT_PITCH, XT_LOW, x_row + 16 * r + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[r][c][e] = __builtin_fmaf(f.x_beta, old[e], f.x_alpha * x[r][c][e]);
                }
            if (p.last && k == p.steps - 1) {
                const int es = c_elem_bytes(a.o_type);
                char* o = (char*)a.o + (entry * a.stride_o + col0 * (p.tall ? a.ldo : 1)) * es;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int n = x_row + 16 * r + 4 * g + e, m = x_col + 16 * c + i;
                            if (n < p.n && m < cols) store_c_any(o + (p.tall ? m * a.ldo + n : n * a.ldo + m) * es, a.o_type, x[r][c][e]);
                        }
                return;
            }
            __syncthreads();  // (T and X have been read)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int n = x_row + 16 * r + 4 * g, m = x_col + 16 * c + i;
                    unsigned w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = split(x[r][c][e]);
                    store4(xt + m * XT_PITCH, XT_LOW, n, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) store1(rg + (n + e) * X_PITCH, X_LOW, m, w[e]);
                }
            __syncthreads();
            sum_s();
        }
        keep();
    }
};

template <int NP, int XT>
__global__ __launch_bounds__(512) void ortho_small_kernel(OrthoSmallArgs p) {
    Small<NP>::template run<XT>(p);
}
template <int NP>
int launch_small(int x_type, const OrthoSmallArgs& p, hipStream_t s) {
    const dim3 grid((unsigned)(p.g.batch * p.chunks));
    switch (x_type) {
    case F16: hipLaunchKernelGGL((ortho_small_kernel<NP, F16>), grid, dim3(512), 0, s, p); break;
    case BF16: hipLaunchKernelGGL((ortho_small_kernel<NP, BF16>), grid, dim3(512), 0, s, p); break;
    default: hipLaunchKernelGGL((ortho_small_kernel<NP, F32>), grid, dim3(512), 0, s, p); break;
    }
    return (int)hipGetLastError();
}

}  // namespace ortho

int launch_ortho_small(int x_type, const OrthoSmallArgs& p, void* stream) {
    return p.n <= 64 ? ortho::launch_small<64>(x_type, p, (hipStream_t)stream) : ortho::launch_small<128>(x_type, p, (hipStream_t)stream);
}

}  // namespace tcm
