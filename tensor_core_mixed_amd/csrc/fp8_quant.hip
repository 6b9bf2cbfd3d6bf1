// Quantiser: a 16- or 32-bit matrix to 8-bit floats with one binary32 scale
// for each block of 128 values of a row, or for each 128 x 128 tile,
//
//     s = max(amax |x| / L, 2^-126),   q = nearest 8-bit value to x / s,
//
// L the format's largest value, so |x| / s never passes it; written as x
// lies, transposed (blocks then run down x's columns), or both from one read.
//
// Every q is the nearest value to the exact quotient, ties to even.
//
// 32-bit inputs: with r = 1/s to an ulp, x r (1 - 2^-21) and x r (1 + 2^-21)
// enclose the exact quotient; where both round to the same 8-bit value (all
// but one element in 10^5) that is the answer.  Where they differ, a middle m
// of two neighbouring values lies between them, and the sign of |x| - |m| s,
// which one fused multiply-add gives exactly, settles it.
//
// 16-bit inputs: both x and amax have few bits, so x L / amax often is a middle
// exactly, and otherwise lies at least 2^-16 away from one.  Where s is amax /
// L rounded up, x / s lies below that middle and x r (1 - 2^-21) rounds as it
// does; where it is rounded down, x r (1 + 2^-21); and where s is exact the
// quotient itself, correctly rounded by one step with its remainder, falls on
// the middle and the conversion takes the even value.  One conversion an
// element, no branch (settling ties as above took three quarters of the waves
// there: 8192^2 bf16 both ways 69 us).
//
// 8192^2 bf16 both ways takes 61.5 us and 4096 x 11008 f32 tiles both ways 53.9:
// 4.4 and 5.0 TB/s, bound by memory (a copy moves 4.86).
//
// NaN and infinity follow the formula: a block that holds a NaN has a NaN
// scale and all q NaN; one with an infinity (and no NaN) has an infinite
// scale, finite x become 0 and the infinities NaN.
//
// Tile kernel: a workgroup takes one 128 x 128 tile, a thread an 8 x 8 block
// of it: 16 lanes read 128 consecutive values of a row (16 bytes a lane for
// 16-bit types), and a thread holds 8 consecutive values in both directions,
// so the bytes of either output pack in registers.  A lane works out one
// row's factors and the 16 lanes of the row share them; a column's go through
// LDS.  Transposed bytes pass through 16 KiB of LDS to be stored 128 bytes of
// a line at a time.  Row kernel: row blocks as they lie need no tile; 16
// lanes take a block, and short matrices fill more of the chip.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace quant {

constexpr int kThreads = 256;
typedef unsigned u2_t __attribute__((ext_vector_type(2)));
typedef unsigned u4_t __attribute__((ext_vector_type(4)));
typedef float f4_t __attribute__((ext_vector_type(4)));

// one step of a maximum over 16 lanes: with the value of the lane ROR places
// away in the row of 16
template <int ROR>
__device__ __forceinline__ unsigned max_ror(unsigned v) {
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROR, 0xf, 0xf, true);
    return v > o ? v : o;
}
__device__ __forceinline__ unsigned max16(unsigned v) {
    return max_ror<1>(max_ror<2>(max_ror<4>(max_ror<8>(v))));
}
__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// |x|'s bits: unsigned order is magnitude order, NaN above infinity
__device__ __forceinline__ unsigned mag(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }
// a maximum that keeps a NaN
__device__ __forceinline__ float max_abs(float m, float v) { return __builtin_elementwise_maximum(m, __builtin_fabsf(v)); }

// amax / L, correctly rounded: the product with 1/L corrected by its
// remainder, which a fused multiply-add gives exactly.
template <bool E5M2>
__device__ __forceinline__ float scale_of(unsigned amax) {
    constexpr float L = E5M2 ? kE5M2Max : kE4M3Max;
    const float x = __builtin_bit_cast(float, amax), q = x * (1.f / L);
    const float s = amax == 0x7f800000u ? x : __builtin_fmaf(__builtin_fmaf(-L, q, x), 1.f / L, q);
    return s < kScaleMin ? kScaleMin : s;  // a NaN stays
}

// What a block's values are multiplied with.  32-bit inputs: the two factors
// that enclose 1/s, and s.  16-bit ones: the factor, and s and 1/s for the
// remainder's step (zeros where it takes none).
struct Factors {
    float a, b, c;
};
template <int XT, bool E5M2>
__device__ __forceinline__ Factors factors_of(float s, unsigned amax) {
    const float r = __builtin_amdgcn_rcpf(s), lo = r * (1.f - 0x1p-21f), hi = r * (1.f + 0x1p-21f);
    if constexpr (XT == F32) {
        return Factors{lo, hi, s};
    } else {
        const float rest = __builtin_fmaf(-(E5M2 ? kE5M2Max : kE4M3Max), s, __builtin_bit_cast(float, amax));
        if (rest == 0.f || s <= kScaleMin) return Factors{r, s, r};  // (the least scale is a power of two)
        return Factors{rest > 0.f ? hi : lo, 0.f, 0.f};
    }
}

// eight values' bytes
template <int XT, bool E5M2>
__device__ __forceinline__ u2_t quant8(const float (&x)[8], const Factors& f) {
    u2_t w;
    if constexpr (XT != F32) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = x[i] * f.a;
            t[i] = __builtin_fmaf(__builtin_fmaf(-t[i], f.b, x[i]), f.c, t[i]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = fp8_encode4<E5M2>(t[4 * h], t[4 * h + 1], t[4 * h + 2], t[4 * h + 3]);
        return w;
    }
    u2_t u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float* v = x + 4 * h;
        w[h] = fp8_encode4<E5M2>(v[0] * f.a, v[1] * f.a, v[2] * f.a, v[3] * f.a);
        u[h] = fp8_encode4<E5M2>(v[0] * f.b, v[1] * f.b, v[2] * f.b, v[3] * f.b);
    }
    if (__ballot(((w[0] ^ u[0]) | (w[1] ^ u[1])) != 0)) {
        const float up = f.c < 0x1p-90f ? 0x1p64f : 1.f;  // (keeps the difference above the least binary32 value)
        const float half = 0.5f * (f.c * up);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned o = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned c0 = (w[h] >> (8 * i)) & 255, c1 = (u[h] >> (8 * i)) & 255;
                const float m2 = fp8_decode<E5M2>(c0) + fp8_decode<E5M2>(c1);
                const float d = __builtin_fmaf(-__builtin_fabsf(m2), half, __builtin_fabsf(x[4 * h + i] * up));
                const unsigned even = (c0 & 1) ? c1 : c0;
                o |= (d > 0.f ? c1 : (d < 0.f ? c0 : even)) << (8 * i);
            }
            w[h] = o;
        }
    }
    return w;
}

// eight consecutive values of a row from p on, of which n exist
template <int XT>
__device__ __forceinline__ void load8(float (&v)[8], const char* p, int64_t n) {
    constexpr int ES = XT == F32 ? 4 : 2;
    if (n >= 8) {
        unsigned w[2 * ES];
        __builtin_memcpy(w, p, 8 * ES);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (XT == F32) v[j] = __builtin_bit_cast(float, w[j]);
            else if constexpr (XT == BF16) v[j] = __builtin_bit_cast(float, (j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
            else v[j] = (float)__builtin_bit_cast(_Float16, (unsigned short)((j & 1) ? w[j >> 1] >> 16 : w[j >> 1]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (n > 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // (values past the row read its last)
                const float x = load_float<XT>(p, min(j, (int)n - 1));
                v[j] = j < n ? x : 0.f;
            }
        }
    }
}

// bytes [0, n) of two words, n <= 8, to any address
__device__ __forceinline__ void store_bytes8(unsigned char* p, u2_t w, int64_t n) {
    if (n >= 8) {
        __builtin_memcpy(p, &w, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (unsigned char)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// lane I of the row of 16 to all of them
template <int I>
__device__ __forceinline__ float row_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_lane(float v, int i) {  // (i a constant once unrolled)
    switch (i) {
    case 0: return row_lane<0>(v);
    case 1: return row_lane<1>(v);
    case 2: return row_lane<2>(v);
    case 3: return row_lane<3>(v);
    case 4: return row_lane<4>(v);
    case 5: return row_lane<5>(v);
    case 6: return row_lane<6>(v);
    default: return row_lane<7>(v);
    }
}

template <int XT, bool E5M2, bool TILE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4))) void quant_tile_kernel(QuantArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2;
    __shared__ u2_t tr[128 * 16];        // transposed bytes: [column][8-byte piece ^ (column / 8)]; before them
                                         // each row group's column maxima, [row group][column]
    __shared__ float fa[128], fb[128], fc[128];  // the columns' factors
    __shared__ unsigned part[4];
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15, wave = tid >> 6;
    const int64_t bc = blockIdx.x, br = blockIdx.y;
    const int64_t row0 = br * 128 + 8 * rg, col0 = bc * 128 + 8 * cg;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        load8<XT>(v[i], (const char*)a.x + ((row0 + i) * a.ldx + col0) * ES, row0 + i < a.rows ? a.cols - col0 : 0);

    float rmax[8], cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (TILE || a.q) rmax[i] = max_abs(rmax[i], v[i][j]);
            if (!TILE) cmax[j] = max_abs(cmax[j], v[i][j]);
        }

    float s_tile = 0.f;
    Factors r_tile{};
    if constexpr (TILE) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, mag(rmax[i]));
        m = max16(m);
        m = umax(m, __shfl_xor(m, 16));
        m = umax(m, __shfl_xor(m, 32));
        if ((tid & 63) == 0) part[wave] = m;
        __syncthreads();
        m = umax(umax(part[0], part[1]), umax(part[2], part[3]));
        s_tile = scale_of<E5M2>(m);
        r_tile = factors_of<XT, E5M2>(s_tile, m);
        if (tid == 0) {
            if (a.q) a.s[br * a.lds + bc] = s_tile;
            if (a.qt) a.st[bc * a.ldst + br] = s_tile;
        }
    } else if (a.qt) {
        f4_t* o = (f4_t*)tr + rg * 32 + 2 * cg;
        o[0] = f4_t{cmax[0], cmax[1], cmax[2], cmax[3]};
        o[1] = f4_t{cmax[4], cmax[5], cmax[6], cmax[7]};
        __syncthreads();
        if (tid < 128) {
            float m = 0.f;
#pragma unroll
            for (int g = 0; g < 16; ++g) m = max_abs(m, ((const float*)tr)[g * 128 + tid]);
            const float s = scale_of<E5M2>(mag(m));
            const Factors r = factors_of<XT, E5M2>(s, mag(m));
            fa[tid] = r.a;
            fb[tid] = r.b;
            fc[tid] = r.c;
            if (bc * 128 + tid < a.cols) a.st[br * a.ldst + bc * 128 + tid] = s;
        }
        __syncthreads();
    }

    if (a.q) {
        // lane i of a row of 16 (and i + 8) works out row i's scale and factors
        float s = s_tile;
        Factors r = r_tile;
        if constexpr (!TILE) {
            unsigned m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const unsigned x = max16(mag(rmax[i]));
                m = (cg & 7) == i ? x : m;
            }
            s = scale_of<E5M2>(m);
            r = factors_of<XT, E5M2>(s, m);
            if (cg < 8 && row0 + cg < a.rows) a.s[bc * a.lds + row0 + cg] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u2_t w = quant8<XT, E5M2>(v[i], TILE ? r : Factors{row_lane(r.a, i), row_lane(r.b, i), row_lane(r.c, i)});
            if (row0 + i < a.rows) store_bytes8(a.q + (row0 + i) * a.ldq + col0, w, a.cols - col0);
        }
    }
    if (!a.qt) return;

#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = v[i][j];
        const int x = 8 * cg + j;
        tr[x * 16 + (rg ^ cg)] = quant8<XT, E5M2>(c, TILE ? r_tile : Factors{fa[x], fb[x], fc[x]});
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = (tid >> 3) + 32 * i, p = tid & 7, x = c >> 3;  // column c, rows 16p .. 16p + 15 of the tile
        const u4_t w = *(const u4_t*)&tr[c * 16 + 2 * (p ^ (x >> 1))];
        const u2_t w0 = (x & 1) ? u2_t{w[2], w[3]} : u2_t{w[0], w[1]}, w1 = (x & 1) ? u2_t{w[0], w[1]} : u2_t{w[2], w[3]};
        const int64_t col = bc * 128 + c, row = br * 128 + 16 * p;
        if (col >= a.cols || row >= a.rows) continue;
        unsigned char* o = a.qt + col * a.ldqt + row;
        if (row + 16 <= a.rows) {
            const u4_t ww = {w0[0], w0[1], w1[0], w1[1]};
            __builtin_memcpy(o, &ww, 16);
        } else {
            store_bytes8(o, w0, a.rows - row);
            if (row + 8 < a.rows) store_bytes8(o + 8, w1, a.rows - row - 8);
        }
    }
}

// Row blocks as they lie: 16 lanes a block, the blocks of 16 rows a workgroup.
template <int XT, bool E5M2>
__global__ __launch_bounds__(kThreads) void quant_row_kernel(QuantArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2;
    const int cg = threadIdx.x & 15;
    const int64_t bc = blockIdx.x, row = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4), col0 = bc * 128 + 8 * cg;
    const char* p = (const char*)a.x + (row * a.ldx + col0) * ES;
    const int64_t n = row < a.rows ? a.cols - col0 : 0;
    float v[8];
    load8<XT>(v, p, n);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_abs(m, v[j]);
    const unsigned amax = max16(mag(m));
    const float s = scale_of<E5M2>(amax);
    const u2_t w = quant8<XT, E5M2>(v, factors_of<XT, E5M2>(s, amax));
    if (n <= 0) return;
    if (cg == 0) a.s[bc * a.lds + row] = s;
    store_bytes8(a.q + row * a.ldq + col0, w, n);
}

template <int XT>
int launch_x(bool e5m2, bool tile, const QuantArgs& a, hipStream_t s) {
    const bool rows_only = !tile && !a.qt;
    const int64_t high = rows_only ? 16 : 128;
    const int64_t nc = scale_blocks(a.cols), nr = (a.rows + high - 1) / high;
    // the grid's y extent holds 65535 workgroups and its x extent 2^32 - 1 threads: larger matrices go in bands
    constexpr int64_t kWide = (int64_t)1 << 23, kHigh = 65535;
    for (int64_t b = 0; b < nr; b += kHigh)
        for (int64_t d = 0; d < nc; d += kWide) {
            QuantArgs e = a;
            const int64_t r0 = b * high, c0 = d * kScaleBlock;
            const int64_t n = nr - b < kHigh ? nr - b : kHigh, m = nc - d < kWide ? nc - d : kWide;
            e.rows = a.rows - r0 < n * high ? a.rows - r0 : n * high;
            e.cols = a.cols - c0 < m * kScaleBlock ? a.cols - c0 : m * kScaleBlock;
            e.x = (const char*)a.x + (r0 * a.ldx + c0) * (XT == F32 ? 4 : 2);
            if (a.q) e.q = a.q + r0 * a.ldq + c0, e.s = a.s + (tile ? b * a.lds + d : d * a.lds + r0);
            if (a.qt) e.qt = a.qt + c0 * a.ldqt + r0, e.st = a.st + (tile ? d * a.ldst + b : b * a.ldst + c0);
            const dim3 grid((unsigned)m, (unsigned)n);
            if (rows_only) {
                if (e5m2) hipLaunchKernelGGL((quant_row_kernel<XT, true>), grid, dim3(kThreads), 0, s, e);
                else hipLaunchKernelGGL((quant_row_kernel<XT, false>), grid, dim3(kThreads), 0, s, e);
            } else if (e5m2) {
                if (tile) hipLaunchKernelGGL((quant_tile_kernel<XT, true, true>), grid, dim3(kThreads), 0, s, e);
                else hipLaunchKernelGGL((quant_tile_kernel<XT, true, false>), grid, dim3(kThreads), 0, s, e);
            } else {
                if (tile) hipLaunchKernelGGL((quant_tile_kernel<XT, false, true>), grid, dim3(kThreads), 0, s, e);
                else hipLaunchKernelGGL((quant_tile_kernel<XT, false, false>), grid, dim3(kThreads), 0, s, e);
            }
        }
    return (int)hipGetLastError();
}

}  // namespace quant

int launch_quantize(int x_type, bool e5m2, bool tile, const QuantArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return quant::launch_x<F16>(e5m2, tile, a, s);
    case BF16: return quant::launch_x<BF16>(e5m2, tile, a, s);
    default: return quant::launch_x<F32>(e5m2, tile, a, s);
    }
}

}  // namespace tcm
