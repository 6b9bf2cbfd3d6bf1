// Quantiser: a 16- or 32-bit matrix to 4-bit floats (e2m1: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives) with a power of two for each block of 32
// values of a row,
//
//     e = clamp(floor(log2 amax |x|) - 2, -127, 127),
//     q = nearest value to x / 2^e, ties to even, 6 for what lies above,
//
// written as x lies, transposed (blocks then run down x's columns), or both
// from one read; and its inverse, x = q 2^e.
//
// floor(log2 amax) is amax's exponent field, so a scale costs a shift and a
// subtraction, and 2 below the field's least value the clamp (a subnormal
// amax, as a block of zeros, has the least scale).  x / 2^e is exact, and the
// hardware's conversion divides, rounds and saturates in one step.  16-bit
// inputs stay packed in pairs from the load to the conversion.
//
// A block that holds a NaN or an infinity has the scale NaN (255) and zeros.
//
// Tile kernel: a workgroup takes one 128 x 128 tile, a thread an 8 x 8 block
// of it.  A row's block of 32 is four lanes, a column's the four rows of
// lanes of one wave, so no maximum leaves a wave.  Transposed values pass
// through LDS to be stored 64 bytes of a column at a time.  Row kernel: row
// blocks as they lie need no tile; short matrices fill more of the chip.
//
// Row blocks run at a copy's rate: 8003 x 8192 bf16 36 us (166 MB, 4.7 TB/s),
// binary32 63 (297 MB); back from rows 25.  Both outputs do not: 64 us from
// HBM (201 MB, 3.1 TB/s; 48 with x in the caches), binary32 102 (333 MB).  A
// tile is loaded, encoded and stored by 3.7 waves a SIMD with none of the next
// one in flight: waves wait for memory in 48% of their cycles and for a turn
// to issue in 39%, the vector ALU is busy in a third.  Back from columns with
// odd pitches 37, whose 16-byte stores lie across lines.  16 x 4096: 2.4 us.
// A tile of 256 x 256 by 1024 threads took 52 us for 48 (binary32 109 for 71,
// x in the caches); for odd pitches stores aligned row by row 82 for 37,
// workgroups of two or four longer pieces of rows 44.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace mxq {

constexpr int kThreads = 256;
typedef unsigned u4_t __attribute__((ext_vector_type(4)));
typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));

// Eight consecutive values: packed pairs, or binary32.
template <int XT>
constexpr int kWords = XT == F32 ? 8 : 4;
template <int XT>
struct Eight {
    unsigned w[kWords<XT>];
};

template <int XT>
__device__ __forceinline__ Eight<XT> load8(const char* p, int64_t n) {
    Eight<XT> v;
    if (n >= 8) {
        __builtin_memcpy(v.w, p, sizeof v.w);
        return v;
    }
#pragma unroll
    for (int i = 0; i < kWords<XT>; ++i) v.w[i] = 0;
    if (n > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // (values past the row read its last)
            const int at = min(j, (int)n - 1);
            if constexpr (XT == F32) {
                unsigned x;
                __builtin_memcpy(&x, p + 4 * at, 4);
                if (j < n) v.w[j] = x;
            } else {
                unsigned short x;
                __builtin_memcpy(&x, p + 2 * at, 2);
                if (j < n) v.w[j >> 1] |= (unsigned)x << (16 * (j & 1));
            }
        }
    }
    return v;
}

// the larger magnitude's bits (in each half, for pairs); a NaN's are the largest
template <int XT>
__device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    if constexpr (XT == F32) return a > b ? a : b;
    else return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(us2_t, a), __builtin_bit_cast(us2_t, b)));
}
template <int XT>
__device__ __forceinline__ unsigned magnitude(unsigned w) {
    return w & (XT == F32 ? 0x7fffffffu : 0x7fff7fffu);
}
// the scale's byte for a block of this amax (one value's bits)
template <int XT>
__device__ __forceinline__ unsigned exponent_of(unsigned amax) {
    unsigned b = amax;
    if constexpr (XT == BF16) b = amax << 16;
    if constexpr (XT == F16) b = __builtin_bit_cast(unsigned, (float)__builtin_bit_cast(_Float16, (unsigned short)amax));
    const int top = (int)(b >> 23);
    return top == 255 ? 255u : (unsigned)max(top - 2, 0);
}
template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// over four neighbouring lanes (quad_perm 1,0,3,2 and 2,3,0,1)
template <int XT>
__device__ __forceinline__ unsigned larger4(unsigned v) {
    v = larger<XT>(v, dpp<0xb1>(v));
    return larger<XT>(v, dpp<0x4e>(v));
}
// the larger half of a pair
template <int XT>
__device__ __forceinline__ unsigned one_of(unsigned v) {
    if constexpr (XT == F32) return v;
    else return larger<XT>(v, v >> 16) & 0xffffu;
}
// a byte of each quad of 16 lanes into a word, the first quad's lowest
__device__ __forceinline__ unsigned gather4(unsigned byte, int quad) {
    unsigned w = byte << (8 * quad);
    w |= dpp<0x124>(w);  // (from the lane 4 and then 8 places away in the 16)
    return w | dpp<0x128>(w);
}

// two values' codes into byte I of w
template <int XT, int I>
__device__ __forceinline__ unsigned encode2(unsigned w, unsigned pair, float scale) {
    if constexpr (XT == BF16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf2_t, pair), scale, I);
    else return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(h2_t, pair), scale, I);
}
template <int I>
__device__ __forceinline__ unsigned encode2(unsigned w, unsigned a, unsigned b, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __builtin_bit_cast(float, a), __builtin_bit_cast(float, b), scale, I);
}
// eight values' codes, the first lowest; zeros under a NaN scale
template <int XT>
__device__ __forceinline__ unsigned encode8(const Eight<XT>& v, unsigned e) {
    const float scale = __builtin_bit_cast(float, e << 23);
    unsigned w = 0;
    if constexpr (XT == F32) {
        w = encode2<0>(w, v.w[0], v.w[1], scale);
        w = encode2<1>(w, v.w[2], v.w[3], scale);
        w = encode2<2>(w, v.w[4], v.w[5], scale);
        w = encode2<3>(w, v.w[6], v.w[7], scale);
    } else {
        w = encode2<XT, 0>(w, v.w[0], scale);
        w = encode2<XT, 1>(w, v.w[1], scale);
        w = encode2<XT, 2>(w, v.w[2], scale);
        w = encode2<XT, 3>(w, v.w[3], scale);
    }
    return e == 255 ? 0 : w;
}
// column j of eight rows
template <int XT>
__device__ __forceinline__ Eight<XT> column(const Eight<XT> (&r)[8], int j) {
    Eight<XT> c;
    if constexpr (XT == F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c.w[i] = r[i].w[j];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c.w[i] = __builtin_amdgcn_perm(r[2 * i + 1].w[j >> 1], r[2 * i].w[j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
    }
    return c;
}

// n of a word's eight codes, n <= 8, to any address
__device__ __forceinline__ void store_codes(unsigned char* p, unsigned w, int64_t n) {
    if (n >= 7) {
        __builtin_memcpy(p, &w, 4);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (2 * i < n) p[i] = (unsigned char)(w >> (8 * i));
    }
}

template <int XT>
__global__ __launch_bounds__(kThreads) void mx_tile_kernel(MxQuantArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2;
    constexpr int kPitch = 17;  // words of a column: 16 and one, so that the writes of a wave spread over the banks
    __shared__ unsigned tr[128 * kPitch];
    __shared__ unsigned te[128];  // the columns' scale words
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15, wave = tid >> 6;
    // (tiles side by side on one XCD, whose cache joins their halves of Q's lines: 8192 x 8192 bf16 48.1 us to 45.6)
    const int64_t bc = xcd_order(blockIdx.x, gridDim.x), br = blockIdx.y;
    const int64_t row0 = br * 128 + 8 * rg, col0 = bc * 128 + 8 * cg;

    Eight<XT> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = load8<XT>((const char*)a.x + ((row0 + i) * a.ldx + col0) * ES, row0 + i < a.rows ? a.cols - col0 : 0);

    if (a.q) {
        unsigned mine = 0;  // lane i of a row of 16 keeps row i's scale word
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            unsigned m = magnitude<XT>(v[i].w[0]);
#pragma unroll
            for (int k = 1; k < kWords<XT>; ++k) m = larger<XT>(m, magnitude<XT>(v[i].w[k]));
            const unsigned e = exponent_of<XT>(one_of<XT>(larger4<XT>(m)));
            const unsigned w = gather4((bc * 128 + 32 * (cg >> 2)) < a.cols ? e : 0, cg >> 2);
            mine = cg == i ? w : mine;
            const unsigned codes = encode8<XT>(v[i], e);
            if (row0 + i < a.rows && col0 < a.cols) store_codes(a.q + (row0 + i) * a.ldq + col0 / 2, codes, a.cols - col0);
        }
        if (cg < 8 && row0 + cg < a.rows) a.s[bc * a.lds + row0 + cg] = mine;
    }

    unsigned cm[kWords<XT>];
#pragma unroll
    for (int k = 0; k < kWords<XT>; ++k) {
        cm[k] = magnitude<XT>(v[0].w[k]);
#pragma unroll
        for (int i = 1; i < 8; ++i) cm[k] = larger<XT>(cm[k], magnitude<XT>(v[i].w[k]));
        cm[k] = larger<XT>(cm[k], (unsigned)__shfl_xor((int)cm[k], 16));
        cm[k] = larger<XT>(cm[k], (unsigned)__shfl_xor((int)cm[k], 32));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const unsigned m = XT == F32 ? cm[j] : (cm[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        const unsigned e = exponent_of<XT>(m);
        tr[(8 * cg + j) * kPitch + rg] = encode8<XT>(column<XT>(v, j), e);
        if ((rg & 3) == 0) ((unsigned char*)te)[(8 * cg + j) * 4 + wave] = (unsigned char)(br * 128 + 32 * wave < a.rows ? e : 0);
    }
    __syncthreads();
    if (tid < 128 && bc * 128 + tid < a.cols) a.st[br * a.ldst + bc * 128 + tid] = te[tid];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = (tid >> 2) + 64 * i, p = tid & 3;  // column c, rows 32 p .. of the tile
        const unsigned* w = tr + c * kPitch + 4 * p;
        const int64_t col = bc * 128 + c, row = br * 128 + 32 * p;
        if (col >= a.cols || row >= a.rows) continue;
        unsigned char* o = a.qt + col * a.ldqt + row / 2;
        const u4_t x = {w[0], w[1], w[2], w[3]};
        if (row + 31 <= a.rows) {
            __builtin_memcpy(o, &x, 16);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) store_codes(o + 4 * k, x[k], a.rows - row - 8 * k);
        }
    }
}

// Row blocks as they lie: 16 lanes a scale word, two words of eight rows a workgroup.
template <int XT>
__global__ __launch_bounds__(kThreads) void mx_row_kernel(MxQuantArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2;
    const int cg = threadIdx.x & 15;
    const int64_t bc = (int64_t)blockIdx.x * 2 + ((threadIdx.x >> 4) & 1), row = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5);
    const int64_t col0 = bc * 128 + 8 * cg;
    const int64_t n = row < a.rows ? a.cols - col0 : 0;
    const Eight<XT> v = load8<XT>((const char*)a.x + (row * a.ldx + col0) * ES, n);
    unsigned m = magnitude<XT>(v.w[0]);
#pragma unroll
    for (int k = 1; k < kWords<XT>; ++k) m = larger<XT>(m, magnitude<XT>(v.w[k]));
    const unsigned e = exponent_of<XT>(one_of<XT>(larger4<XT>(m)));
    const unsigned word = gather4(bc * 128 + 32 * (cg >> 2) < a.cols ? e : 0, cg >> 2);
    const unsigned codes = encode8<XT>(v, e);
    if (n <= 0) return;
    if (cg == 0) a.s[bc * a.lds + row] = word;
    store_codes(a.q + row * a.ldq + col0 / 2, codes, n);
}

// Back: a thread takes eight values of a row.
template <int XT>
__global__ __launch_bounds__(kThreads) void mx_back_kernel(MxQuantArgs a) {
    constexpr int ES = XT == F32 ? 4 : 2;
    const int cg = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5), col0 = (int64_t)blockIdx.x * 256 + 8 * cg;
    if (row >= a.rows || col0 >= a.cols) return;
    const int64_t n = a.cols - col0;
    const unsigned char* p = a.q + row * a.ldq + col0 / 2;
    unsigned w = 0;
    if (n >= 7) {
        __builtin_memcpy(&w, p, 4);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) w |= 2 * i < n ? (unsigned)p[i] << (8 * i) : 0;
    }
    const unsigned e = (a.s[col0 / 128 * a.lds + row] >> (8 * (int)(col0 / 32 % 4))) & 255;
    const float scale = __builtin_bit_cast(float, e == 255 ? 0x7fc00000u : e << 23);
    char* o = (char*)const_cast<void*>(a.x) + (row * a.ldx + col0) * ES;
    Eight<XT> v;
    if constexpr (XT == F32) {
        f2_t y[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3)};
#pragma unroll
        for (int i = 0; i < 8; ++i) v.w[i] = __builtin_bit_cast(unsigned, e == 255 ? scale : y[i >> 1][i & 1]);
    } else if constexpr (XT == BF16) {
        bf2_t y[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3)};
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = e == 255 ? 0x7fc07fc0u : __builtin_bit_cast(unsigned, y[i]);
    } else {
        h2_t y[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3)};
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = e == 255 ? 0x7e007e00u : __builtin_bit_cast(unsigned, y[i]);
    }
    if (n >= 8) {
        __builtin_memcpy(o, v.w, sizeof v.w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            if constexpr (XT == F32) {
                __builtin_memcpy(o + 4 * j, &v.w[j], 4);
            } else {
                const unsigned short h = (unsigned short)(v.w[j >> 1] >> (16 * (j & 1)));
                __builtin_memcpy(o + 2 * j, &h, 2);
            }
        }
    }
}

// The grid's y extent holds 65535 workgroups and its x extent 2^32 - 1 threads: larger matrices go in bands of
// workgroups of `high` rows by `wide` columns.
template <class F>
int in_bands(const MxQuantArgs& a, int es, int64_t wide, int64_t high, F launch) {
    const int64_t nc = (a.cols + wide - 1) / wide, nr = (a.rows + high - 1) / high;
    constexpr int64_t kWide = (int64_t)1 << 23, kHigh = 65280;  // (kHigh rows of either height are a multiple of 128)
    for (int64_t b = 0; b < nr; b += kHigh)
        for (int64_t d = 0; d < nc; d += kWide) {
            MxQuantArgs e = a;
            const int64_t r0 = b * high, c0 = d * wide;
            const int64_t n = nr - b < kHigh ? nr - b : kHigh, m = nc - d < kWide ? nc - d : kWide;
            e.rows = a.rows - r0 < n * high ? a.rows - r0 : n * high;
            e.cols = a.cols - c0 < m * wide ? a.cols - c0 : m * wide;
            e.x = (const char*)a.x + (r0 * a.ldx + c0) * es;
            if (a.q) e.q = a.q + r0 * a.ldq + c0 / 2, e.s = a.s + c0 / kMxWord * a.lds + r0;
            if (a.qt) e.qt = a.qt + c0 * a.ldqt + r0 / 2, e.st = a.st + r0 / kMxWord * a.ldst + c0;
            launch(e, dim3((unsigned)m, (unsigned)n));
        }
    return (int)hipGetLastError();
}

template <int XT>
int quantize(const MxQuantArgs& a, hipStream_t s) {
    constexpr int ES = XT == F32 ? 4 : 2;
    if (!a.qt)
        return in_bands(a, ES, 256, 8, [&](const MxQuantArgs& e, dim3 grid) {
            hipLaunchKernelGGL(mx_row_kernel<XT>, grid, dim3(kThreads), 0, s, e);
        });
    return in_bands(a, ES, 128, 128, [&](const MxQuantArgs& e, dim3 grid) {
        hipLaunchKernelGGL(mx_tile_kernel<XT>, grid, dim3(kThreads), 0, s, e);
    });
}
template <int XT>
int dequantize(const MxQuantArgs& a, hipStream_t s) {
    return in_bands(a, XT == F32 ? 4 : 2, 256, 8, [&](const MxQuantArgs& e, dim3 grid) {
        hipLaunchKernelGGL(mx_back_kernel<XT>, grid, dim3(kThreads), 0, s, e);
    });
}

}  // namespace mxq

int launch_mx_quantize(int x_type, const MxQuantArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return mxq::quantize<F16>(a, s);
    case BF16: return mxq::quantize<BF16>(a, s);
    default: return mxq::quantize<F32>(a, s);
    }
}
int launch_mx_dequantize(int x_type, const MxQuantArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return mxq::dequantize<F16>(a, s);
    case BF16: return mxq::dequantize<BF16>(a, s);
    default: return mxq::dequantize<F32>(a, s);
    }
}

}  // namespace tcm
