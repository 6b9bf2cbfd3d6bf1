// Quantiser: a 16- or 32-bit matrix to 8-bit floats with one binary32 scale
// for each block of 128 values of a row, or for each 128 x 128 tile,
//
//     s = max(amax |x| / L, 2^-126),   q = nearest 8-bit value to x / s,
//
// L the format's largest value, so |x| / s never passes it; written as x
// lies, transposed (blocks then run down x's columns), or both from one read.
//
// Every q is the nearest value to the exact quotient, ties to even.  With
// r = 1/s to an ulp, x r (1 - 2^-20) and x r (1 + 2^-20) enclose the exact
// quotient; where both round to the same 8-bit value (all but about one
// element in 10^5 of ordinary data) that is the answer, for two
// multiplications and a packed conversion an element.  Where they differ, a
// middle m of two neighbouring values lies between them, and |x| is compared
// with |m| s in binary64, which holds that product exactly.
//
// NaN and infinity follow the formula: a block that holds a NaN has a NaN
// scale and all q NaN; one with an infinity (and no NaN) has an infinite
// scale, finite x become 0 and the infinities NaN.
//
// A workgroup takes one 128 x 128 tile, a thread an 8 x 8 block of it: 16
// lanes read 128 consecutive values of a row (16 bytes a lane for 16-bit
// types), and a thread holds 8 consecutive values in both directions, so the
// bytes of either output pack in registers.  Transposed bytes pass through
// 16 KiB of LDS to be stored 128 bytes of a line at a time.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace quant {

constexpr int kThreads = 256;
typedef unsigned u2_t __attribute__((ext_vector_type(2)));
typedef unsigned u4_t __attribute__((ext_vector_type(4)));

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

template <bool E5M2>
__device__ __forceinline__ float scale_of(unsigned amax) {
    const float s = __builtin_bit_cast(float, amax) / (E5M2 ? kE5M2Max : kE4M3Max);
    return s < kScaleMin ? kScaleMin : s;  // a NaN stays
}

// the two factors that enclose 1/s
struct Recip {
    float lo, hi;
};
__device__ __forceinline__ Recip recip_of(float s) {
    const float r = __builtin_amdgcn_rcpf(s);
    return Recip{r * (1.f - 0x1p-20f), r * (1.f + 0x1p-20f)};
}

// a byte of which the enclosing quotients disagree
template <bool E5M2>
__device__ __forceinline__ unsigned settle(unsigned c0, unsigned c1, float x, float s) {
    if (c0 == c1) return c0;
    const double m = 0.5 * ((double)fp8_decode<E5M2>(c0) + (double)fp8_decode<E5M2>(c1));
    const double d = fabs((double)x) - fabs(m) * (double)s;
    return d > 0 ? c1 : (d < 0 ? c0 : ((c0 & 1) ? c1 : c0));
}
template <bool E5M2>
__device__ __forceinline__ unsigned quant4(const float (&x)[4], const float (&s)[4], const Recip (&r)[4]) {
    unsigned lo = fp8_encode4<E5M2>(x[0] * r[0].lo, x[1] * r[1].lo, x[2] * r[2].lo, x[3] * r[3].lo);
    const unsigned hi = fp8_encode4<E5M2>(x[0] * r[0].hi, x[1] * r[1].hi, x[2] * r[2].hi, x[3] * r[3].hi);
    if (lo != hi) {
        unsigned w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= settle<E5M2>((lo >> (8 * i)) & 255, (hi >> (8 * i)) & 255, x[i], s[i]) << (8 * i);
        lo = w;
    }
    return lo;
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

template <int XT, bool E5M2, bool TILE>
__global__ __launch_bounds__(kThreads) void quant_kernel(QuantArgs a) {
    __shared__ u2_t tr[128 * 16];        // transposed bytes: [column][8-byte piece ^ (column / 8)]
    __shared__ unsigned part[4][128];    // each wave's column maxima; row 0 the tile's with TILE
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15, wave = tid >> 6;
    const int64_t bc = blockIdx.x, br = blockIdx.y;
    const int64_t row0 = br * 128 + 8 * rg, col0 = bc * 128 + 8 * cg;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = row0 + i < a.rows;
        constexpr int ES = XT == F32 ? 4 : 2;
        const char* p = (const char*)a.x + ((row0 + i) * a.ldx + col0) * ES;
        if (in && col0 + 8 <= a.cols) {
            unsigned w[2 * ES];
            __builtin_memcpy(w, p, 8 * ES);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (XT == F32) v[i][j] = __builtin_bit_cast(float, w[j]);
                else if constexpr (XT == BF16) v[i][j] = __builtin_bit_cast(float, (j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
                else v[i][j] = (float)__builtin_bit_cast(_Float16, (unsigned short)((j & 1) ? w[j >> 1] >> 16 : w[j >> 1]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = in && col0 + j < a.cols ? load_float<XT>(p, j) : 0.f;
        }
    }

    unsigned rmax[8], cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned m = mag(v[i][j]);
            rmax[i] = umax(rmax[i], m);
            cmax[j] = umax(cmax[j], m);
        }

    float s_tile = 0.f;
    if constexpr (TILE) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, rmax[i]);
        m = max16(m);
        m = umax(m, __shfl_xor(m, 16));
        m = umax(m, __shfl_xor(m, 32));
        if ((tid & 63) == 0) part[0][wave] = m;
        __syncthreads();
        m = umax(umax(part[0][0], part[0][1]), umax(part[0][2], part[0][3]));
        s_tile = scale_of<E5M2>(m);
        if (tid == 0) {
            if (a.q) a.s[br * a.lds + bc] = s_tile;
            if (a.qt) a.st[bc * a.ldst + br] = s_tile;
        }
    }

    if (a.q) {
        float keep = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = TILE ? s_tile : scale_of<E5M2>(max16(rmax[i]));
            const Recip r = recip_of(s);
            if (cg == i) keep = s;
            u2_t w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = quant4<E5M2>({v[i][4 * h], v[i][4 * h + 1], v[i][4 * h + 2], v[i][4 * h + 3]}, {s, s, s, s}, {r, r, r, r});
            if (row0 + i < a.rows) store_bytes8(a.q + (row0 + i) * a.ldq + col0, w, a.cols - col0);
        }
        if (!TILE && cg < 8 && row0 + cg < a.rows) a.s[bc * a.lds + row0 + cg] = keep;
    }
    if (!a.qt) return;

    float sc[8];
    Recip rc[8];
    if constexpr (!TILE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cmax[j] = umax(cmax[j], __shfl_xor(cmax[j], 16));
            cmax[j] = umax(cmax[j], __shfl_xor(cmax[j], 32));
        }
        if ((tid & 63) < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) part[wave][8 * cg + j] = cmax[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * cg + j;
            sc[j] = scale_of<E5M2>(umax(umax(part[0][c], part[1][c]), umax(part[2][c], part[3][c])));
        }
        if (rg == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col0 + j < a.cols) a.st[br * a.ldst + col0 + j] = sc[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = s_tile;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) rc[j] = recip_of(sc[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u2_t w;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = quant4<E5M2>({v[4 * h][j], v[4 * h + 1][j], v[4 * h + 2][j], v[4 * h + 3][j]}, {sc[j], sc[j], sc[j], sc[j]},
                                {rc[j], rc[j], rc[j], rc[j]});
        tr[(8 * cg + j) * 16 + (rg ^ cg)] = w;
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

template <int XT>
int launch_x(bool e5m2, bool tile, const QuantArgs& a, hipStream_t s) {
    const int64_t nc = scale_blocks(a.cols), nr = scale_blocks(a.rows);
    // the grid's y extent holds 65535 tiles: longer matrices go in bands
    for (int64_t b = 0; b < nr; b += 65535) {
        QuantArgs e = a;
        const int64_t r0 = b * 128;
        e.rows = a.rows - r0;
        e.x = (const char*)a.x + r0 * a.ldx * (XT == F32 ? 4 : 2);
        if (a.q) e.q = a.q + r0 * a.ldq, e.s = a.s + (tile ? b * a.lds : r0);
        if (a.qt) e.qt = a.qt + r0, e.st = a.st + (tile ? b : b * a.ldst);
        const int64_t n = nr - b < 65535 ? nr - b : 65535;
        if (n * 128 < e.rows) e.rows = n * 128;
        const dim3 grid((unsigned)nc, (unsigned)n);
        if (e5m2) {
            if (tile) hipLaunchKernelGGL((quant_kernel<XT, true, true>), grid, dim3(kThreads), 0, s, e);
            else hipLaunchKernelGGL((quant_kernel<XT, true, false>), grid, dim3(kThreads), 0, s, e);
        } else {
            if (tile) hipLaunchKernelGGL((quant_kernel<XT, false, true>), grid, dim3(kThreads), 0, s, e);
            else hipLaunchKernelGGL((quant_kernel<XT, false, false>), grid, dim3(kThreads), 0, s, e);
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
