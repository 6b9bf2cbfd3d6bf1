// Tiled kernel of the block-scaled 8-bit product,
//
//     C[m][n] = epi(init + sum over blocks b of 128 k of
//                          (sa[b][m] * sb[b, n]) * P_b[m][n]),
//     P_b[m][n] = sum over the block's k of A[m][k] * B[n][k].
//
// One scale block is one K-step and one matrix instruction deep: a
// 16x16x128 8-bit MFMA with a zero accumulator gives P_b of a 16 x 16 tile
// whole, and four multiply-adds a lane add it, scaled, to the binary32
// accumulator while the next MFMA runs (the MFMA holds the matrix core for 32
// cycles, the multiply-adds the vector ALU for 16; with a scale of its own for
// every row of B the factor is one more multiplication each, 32).  The MFMA's
// own block exponents are not used: the scales are arbitrary binary32 values.
// The two scales are multiplied first, once for sixteen values of a lane: to
// multiply the sum by one after the other would double the multiply-adds, and
// differs only where the scales' product leaves binary32's normal range.
//
// The MFMA takes its A operand from B's rows and its B operand from A's, so a
// lane's accumulators run along n at one m: sa is one value a lane and tile,
// and a row's stores are contiguous: row i of a wave's tiles j = 0 .. 3 is
// column 16 (i / 4) + 4 j + i % 4 of its 64 for 16-bit C (16 columns, 32 bytes
// a lane) and 16 j + i for binary32 C (four lanes write 64 bytes together:
// 8039x7376x1504 225 us, 248 with the other order; 16-bit C was 1% slower).
// (Which k an operand register holds plays no part as long as both operands
// agree.)
//
// Copies, LDS layout and pipeline are the dense kernels': 128-byte rows of
// each operand go to LDS by 16-byte direct loads, the chunk index XOR-ed with
// a function of the row so that the reads of a fragment fall on distinct
// banks; STAGES stages, copies STAGES - 1 steps ahead.  The scales of a step
// travel with it (4-byte direct loads).
//
// 8192^3 takes 460 to 475 us (2.3 to 2.4 PFLOP/s; the matrix cores 61% busy at
// 1.85 GHz; 348 us without the copies, 448 without the multiply-adds), f32 C
// 4096x4096x5003 with two row scales 167 us (1.0 PFLOP/s, bound by the vector
// ALU: a tile's four 16-bit MFMAs come with eight conversions, four products
// of two scales and four multiply-adds a lane).
#pragma once
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace fp8t {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_void;

constexpr unsigned kOOB = 0x40000000u;  // past every descriptor's range: such loads give zeros
constexpr int kRsrcWord3 = 0x00020000;  // raw dword access

// bytes [0, n) of a chunk, the others zero
__device__ __forceinline__ i4 keep_bytes(i4 v, int n) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int k = n - 4 * d;
        v[d] = k >= 4 ? v[d] : (k <= 0 ? 0 : (int)((unsigned)v[d] & (0xffffffffu >> (32 - 8 * k))));
    }
    return v;
}

// One lane's 32 bytes of an operand as the matrix instruction takes them: the
// bytes themselves, or (WIDE) 16-bit floats, which hold both formats exactly.
template <bool WIDE>
struct Operand {
    i8v v;
};
template <>
struct Operand<true> {
    h8 v[4];
};
template <bool E5, bool WIDE>
__device__ __forceinline__ Operand<WIDE> operand(i8v x) {
    Operand<WIDE> o;
    if constexpr (!WIDE) {
        o.v = x;
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) o.v[q] = fp8_to_f16x8<E5>(x[2 * q], x[2 * q + 1]);
    }
    return o;
}
// The sum of 128 products.  8-bit operands are taken where C has 16 bits: their instruction cuts products 13 bits below the
// largest of each eight, off by 2^-16 of C's average size on average (1/32 of half a step of f16, 1/256 of bf16's) at
// twice the rate.  Binary32 C takes the 16-bit operands, whose sums are binary32 ones.
template <bool A5, bool B5, bool WIDE>
__device__ __forceinline__ f4 mma(const Operand<WIDE>& b, const Operand<WIDE>& a) {
    f4 p = {0.f, 0.f, 0.f, 0.f};
    if constexpr (!WIDE) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, p, B5 ? 1 : 0, A5 ? 1 : 0, 0, 0, 0, 0);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[q], a.v[q], p, 0, 0, 0);
        return p;
    }
}

// E consecutive columns n .. of rows of C
template <int E>
struct Epilogue {
    const Fp8Args& a;
    int64_t n;
    bool full;  // all of them exist
    float bias[E];

    __device__ __forceinline__ Epilogue(const Fp8Args& a, int64_t n) : a(a), n(n), full(n + E <= a.N) {
        if (a.has_bias) {
#pragma unroll
            for (int j = 0; j < E; ++j) bias[j] = a.bias[min(n + j, a.N - 1)];
        }
    }
    // v += row m of C
    __device__ __forceinline__ void add_c(float (&v)[E], const char* c) const {
        if (full && a.c_vec) {
            if (a.c_type == C_ACC) {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const f4 x = *(const f4*)(c + 16 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[4 * q + i] += x[i];
                }
            } else {
                unsigned w[E / 2];
                __builtin_memcpy(w, __builtin_assume_aligned(c, E >= 8 ? 16 : 8), 2 * E);
#pragma unroll
                for (int q = 0; q < E; ++q) {
                    const unsigned short h = (unsigned short)(w[q >> 1] >> (16 * (q & 1)));
                    v[q] += a.c_type == C_F16 ? (float)__builtin_bit_cast(_Float16, h) : __builtin_bit_cast(float, (unsigned)h << 16);
                }
            }
        } else {
            const int cs = c_elem_bytes(a.c_type);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] += load_c_any(c + min<int64_t>(j, a.N - 1 - n) * cs, a.c_type);
        }
    }
    // v + bias + C's contents, ReLU, stored in C's type as row m
    __device__ __forceinline__ void store(float (&v)[E], int64_t m) const {
        char* c = (char*)a.C + (m * a.ldc + n) * c_elem_bytes(a.c_type);
        if (a.has_bias) {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] += bias[j];
        }
        if (a.accum) add_c(v, c);
        if (a.relu) {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = v[j] > 0.f ? v[j] : 0.f;
        }
        if (full && a.c_vec) {
            if (a.c_type == C_ACC) {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) *(f4*)(c + 16 * q) = f4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            } else {
                unsigned w[E / 2];
#pragma unroll
                for (int q = 0; q < E / 2; ++q) {
                    unsigned lo, hi;
                    if (a.c_type == C_F16) {
                        lo = __builtin_bit_cast(unsigned short, (_Float16)v[2 * q]);
                        hi = __builtin_bit_cast(unsigned short, (_Float16)v[2 * q + 1]);
                    } else {
                        lo = __builtin_bit_cast(unsigned short, (__bf16)v[2 * q]);
                        hi = __builtin_bit_cast(unsigned short, (__bf16)v[2 * q + 1]);
                    }
                    w[q] = lo | hi << 16;
                }
                __builtin_memcpy(__builtin_assume_aligned(c, E >= 8 ? 16 : 8), w, 2 * E);
            }
        } else {
            const int cs = c_elem_bytes(a.c_type);
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (n + j < a.N) store_c_any(c + j * cs, a.c_type, v[j]);
        }
    }
};

template <int CFG, bool A5, bool B5, bool BROW, bool WIDE>
struct Tile {
    static constexpr Fp8Tile cfg = kFp8Tiles[CFG];
    static constexpr int BM = cfg.bm, BN = cfg.bn, WM = cfg.wm, WN = cfg.wn, NST = cfg.stages;
    static constexpr int NW = WM * WN, NT = NW * 64;
    static constexpr int TM = BM / WM, FM = TM / 16;  // 16-row tiles of A a wave
    static_assert(BN / WN == 64, "a wave covers 64 columns");
    static constexpr int GM = FM >= 4 ? 2 : 1, NG = FM / GM;        // row tiles taken together, groups a K-step
    static_assert(FM % (2 * GM) == 0, "a step starts with the first of the two fragment buffers");
    static_assert(NW == 8 || NW == 4, "");
    static constexpr int IA = BM / (8 * NW), IB = BN / (8 * NW);
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + 1024;
    static constexpr int STAGE = SB_OFF + 1024;
    static constexpr int LDS = NST * STAGE;
    static_assert(LDS <= 160 * 1024 && BM <= 256 && BN <= 256, "");

    // The column of the wave's 64 that is row i of its tile j, and its parts: n_row(i) + n_tile(j).
    __device__ __forceinline__ static constexpr int n_row(int i) { return WIDE ? i : 16 * (i >> 2) + (i & 3); }
    __device__ __forceinline__ static constexpr int n_tile(int j) { return (WIDE ? 16 : 4) * j; }
    // Both swizzles of the row that a fragment read takes as its i-th are i / 2 % 8: any sixteen lanes that the LDS serves
    // at once (0-3, 12-15, 20-27 and their complements, by the counters) then fall on distinct banks.  (With i % 8 ^ i / 8
    // for A every read of A took twice its time.)
    __device__ __forceinline__ static int swz_a(int r) { return (r >> 1) & 7; }
    __device__ __forceinline__ static int swz_b(int r) { return WIDE ? (r >> 1) & 7 : ((r >> 1) & 1) | ((r >> 4) & 3) << 1; }

    // A wave's copies of a step: IA of A, IB of B, and of the scales one (eight waves: 0-3 A's and 4-7 B's) or two.
    static constexpr int NS = NW == 4 ? 2 : 1, OPS = IA + IB + NS;
    // this lane's offsets in them, and where the next step to copy begins
    struct Dma {
        unsigned a_off, b_off[2], s_off[NS];
        int a_k, b_k[2];
        const unsigned char *pa, *pb;
        const float* ps[NS];
        int64_t s_step[NS];  // floats
        int s_lds[NS];
        unsigned a_hop, b_hop;
        int a_range, b_range, k_left, steps_left;
        // of the step being copied: offsets, out of range past its data, and ranges, empty past the last step.  (The
        // range is checked against the lane's offset alone, so the whole of it goes there.)
        unsigned oa, ob[2], os[NS];
        int ra, rb;
    };
    __device__ __forceinline__ static void dma_setup(Dma& d, const Fp8Args& a, int64_t m0, int64_t n0, int k_lo, int k_hi, int wave,
                                                     int lane) {
        {
            const int r = 8 * wave + (lane >> 3), c = (lane & 7) ^ swz_a(r);
            d.a_off = (unsigned)(r * (int)a.lda + 16 * c);
            d.a_k = 16 * c;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // (with four waves the swizzle of rows 32 apart differs: two offsets)
            const int r = 8 * (NW * q + wave) + (lane >> 3), c = (lane & 7) ^ swz_b(r);
            d.b_off[q] = (unsigned)(r * (int)a.ldb + 16 * c);
            d.b_k[q] = 16 * c;
        }
        const int i = 64 * (wave & 3) + lane;
        const unsigned sa_off = i < BM && m0 + i < a.M ? (unsigned)(4 * i) : kOOB;
        const unsigned sb_off =
            i >= BN || n0 + i >= a.N ? kOOB : (BROW ? (unsigned)(4 * i) : (unsigned)(((i + (int)(n0 & 127)) >> 7) * (int)a.ldsb * 4));
        const float* psa = a.sa + k_lo * a.ldsa + m0;
        const float* psb = BROW ? a.sb + k_lo * a.ldsb + n0 : a.sb + n0 / 128 * a.ldsb + k_lo;
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            const bool of_b = NS == 2 ? q == 1 : wave >= 4;
            d.s_off[q] = of_b ? sb_off : sa_off;
            d.ps[q] = of_b ? psb : psa;
            d.s_step[q] = of_b ? (BROW ? a.ldsb : 1) : a.ldsa;
            d.s_lds[q] = (of_b ? SB_OFF : SA_OFF) + (wave & 3) * 256;
        }
        const int64_t k0 = (int64_t)k_lo * 128;
        d.pa = a.A + m0 * a.lda + k0;
        d.pb = a.B + n0 * a.ldb + k0;
        d.a_hop = (unsigned)(8 * NW * (int)a.lda);
        d.b_hop = (unsigned)(16 * NW * (int)a.ldb);
        // the ranges end with the last row's last 16-byte chunk (which may hold bytes past K)
        const int left = (int)(a.K - k0);
        const int rows_a = min((int)a.M - (int)m0, BM), rows_b = min((int)a.N - (int)n0, BN);
        d.a_range = (rows_a - 1) * (int)a.lda + ((left + 15) & ~15);
        d.b_range = (rows_b - 1) * (int)a.ldb + ((left + 15) & ~15);
        d.k_left = left;
        d.steps_left = k_hi - k_lo;
    }
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const void* p, int n) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, kRsrcWord3);
    }
    // Copy `op` of the next step into the stage at s, ops in rising order.  Past the last step the copies run on with
    // every lane out of range (zeros into a stage that is not read again): no branch splits the loop.
    __device__ __forceinline__ static void dma_op(Dma& d, lds_char* s, int op, int wave) {
        if (op == 0) {
            const int left = d.steps_left > 0 ? d.k_left : 0;
            d.ra = left > 0 ? d.a_range : 0;
            d.rb = left > 0 ? d.b_range : 0;
            d.oa = d.a_k < left ? d.a_off : kOOB;
            d.ob[0] = d.b_k[0] < left ? d.b_off[0] : kOOB;
            d.ob[1] = d.b_k[1] < left ? d.b_off[1] : kOOB;
#pragma unroll
            for (int q = 0; q < NS; ++q) d.os[q] = left > 0 ? d.s_off[q] : kOOB;
        }
        if (op < IA) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(d.pa, d.ra), (lds_void*)(s + (NW * op + wave) * 1024), 16, d.oa + op * d.a_hop, 0, 0,
                                                     0);
        } else if (op < IA + IB) {
            const int j = op - IA;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(d.pb, d.rb), (lds_void*)(s + A_BYTES + (NW * j + wave) * 1024), 16,
                                                     d.ob[j & 1] + (j >> 1) * d.b_hop, 0, 0, 0);
        } else {
            const int q = op - IA - IB;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(d.ps[q], (int)kOOB), (lds_void*)(s + d.s_lds[q]), 4, d.os[q], 0, 0, 0);
        }
        if (op == OPS - 1) {
            d.pa += 128;
            d.pb += 128;
#pragma unroll
            for (int q = 0; q < NS; ++q) d.ps[q] += d.s_step[q];
            d.a_range -= 128;
            d.b_range -= 128;
            d.k_left -= 128;
            --d.steps_left;
        }
    }
    // (__syncthreads would wait for the copies in flight)
    __device__ __forceinline__ static void barrier() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // until STEPS K-steps of this wave's copies are in flight, and every LDS read has returned
    template <int STEPS>
    __device__ __forceinline__ static void wait_copies() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(STEPS * OPS) : "memory");
    }

    // The last step of a K that is no multiple of 16: zeros for the bytes past K of the chunk that K ends in.
    __device__ __forceinline__ static void mask_tail(lds_char* smem, int st, int krem, int tid) {
        const int c = krem >> 4;
        for (int r = tid; r < BM + BN; r += NT) {
            const int x = r < BM ? swz_a(r) : swz_b(r - BM);
            __attribute__((address_space(3))) i4* p =
                (__attribute__((address_space(3))) i4*)(smem + st * STAGE + r * 128 + ((c ^ x) << 4));
            *p = keep_bytes(*p, krem & 15);
        }
        __syncthreads();
    }

    struct Lane {
        int a[2], b[2];   // byte offsets within a stage of this lane's two chunks of row tile 0
        int sa, sb;
    };
    __device__ __forceinline__ static i8v read_pair(const lds_char* s, int o0, int o1) {
        const i4 x = *(const __attribute__((address_space(3))) i4*)(s + o0);
        const i4 y = *(const __attribute__((address_space(3))) i4*)(s + o1);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ static float lds_f(const lds_char* s, int o) {
        return *(const __attribute__((address_space(3))) float*)(s + o);
    }

    struct Rows {  // a group of row tiles
        i8v a[GM];
        float s[GM];
    };
    struct Cols {
        i8v b[4];
        f4 s[BROW ? 4 : 1];
    };
    __device__ __forceinline__ static void read_rows(Rows& f, const lds_char* s, const Lane& l, int g) {
#pragma unroll
        for (int i = 0; i < GM; ++i) {
            f.a[i] = read_pair(s, l.a[0] + (g * GM + i) * 2048, l.a[1] + (g * GM + i) * 2048);
            f.s[i] = lds_f(s, l.sa + (g * GM + i) * 64);
        }
    }
    __device__ __forceinline__ static void read_col(Cols& f, const lds_char* s, const Lane& l, int j) {
        f.b[j] = read_pair(s, l.b[0] + n_tile(j) * 128, l.b[1] + n_tile(j) * 128);
    }
    __device__ __forceinline__ static void read_scales(Cols& f, const lds_char* s, const Lane& l) {
        if constexpr (BROW) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f.s[j] = *(const __attribute__((address_space(3))) f4*)(s + l.sb + 4 * n_tile(j));
        } else {
            f.s[0][0] = lds_f(s, l.sb);
        }
    }
    __device__ __forceinline__ static void scale_add(f4& acc, f4 p, float sa, const Cols& f, int j) {
        if constexpr (BROW) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], sa * f.s[j][r], acc[r]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], sa, acc[r]);  // (sa times the tile's scale)
        }
    }

    // (keeps the compiler from sinking multiply-adds past the branches of the pipeline)
    __device__ __forceinline__ static void pin(f4& v) { asm volatile("" : "+v"(v)); }

    // The copies of step kt + NST go out a few at a time, from the last group of step kt (whose stage is then free) into
    // the groups of step kt + 1: sent in one piece they fill the address queue and hold the matrix cores up (8192^3
    // 490 us, spread 465).  With two stages and two groups they have to land within the step: all at once.
    static constexpr int SLOTS = NG >= 4 ? 12 : (NST > 2 ? 8 : 4);
    static constexpr int PER_SLOT = (OPS + SLOTS - 1) / SLOTS;
    __device__ __forceinline__ static void dma_slot(Dma& d, lds_char* s, int slot, int wave) {
#pragma unroll
        for (int i = 0; i < PER_SLOT; ++i)
            if (slot < SLOTS && slot * PER_SLOT + i < OPS) dma_op(d, s, slot * PER_SLOT + i, wave);
    }
    static constexpr int slot_ops(int slot) {
        return slot >= SLOTS || slot * PER_SLOT >= OPS ? 0 : (OPS - slot * PER_SLOT < PER_SLOT ? OPS - slot * PER_SLOT : PER_SLOT);
    }

    struct Pipe {
        Rows fr[2];
        Cols fc;
        int st;
    };
    // One K-step from stage f.st.  MASK: the next one is the matrix's last and K no multiple of 16.
    template <bool MASK>
    __device__ __forceinline__ static void kstep(f4 (&acc)[FM][4], Pipe& f, Dma& d, const Lane& l, lds_char* smem, int k_tail,
                                                 int wave) {
        lds_char* s = smem + f.st * STAGE;
        const int sn = f.st + 1 == NST ? 0 : f.st + 1;
        const lds_char* nx = smem + sn * STAGE;
        lds_char* before = smem + (f.st == 0 ? NST - 1 : f.st - 1) * STAGE;  // the stage of the step before
        f4 p[2][GM];
        float t[2][GM];
        Operand<WIDE> ob[4];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            Rows& cur = f.fr[g & 1];
            Rows& nxt = f.fr[(g + 1) & 1];
            const bool end = g == NG - 1;
#pragma unroll
            for (int i = 0; i < GM; ++i) t[g & 1][i] = BROW ? cur.s[i] : cur.s[i] * f.fc.s[0][0];
            Operand<WIDE> oa[GM];
#pragma unroll
            for (int i = 0; i < GM; ++i) oa[i] = operand<A5, WIDE>(cur.a[i]);
            if (!end) {
                read_rows(nxt, s, l, g + 1);
            } else {
                // every fragment of this step is in registers: the next step's copies must have landed, and those of
                // step kt + NST may overwrite this stage
#pragma unroll
                for (int i = 0; i < FM - GM; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) pin(acc[i][j]);
                wait_copies<NST - 2>();
                barrier();
                if constexpr (MASK) mask_tail(smem, sn, k_tail, threadIdx.x);
                read_rows(nxt, nx, l, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = g * 4 + j, slot = end ? j : 4 + q;
                if (g == 0) ob[j] = operand<B5, WIDE>(f.fc.b[j]);
#pragma unroll
                for (int i = 0; i < GM; ++i) p[q & 1][i] = mma<A5, B5, WIDE>(ob[j], oa[i]);
                if (end) read_col(f.fc, nx, l, j);
                dma_slot(d, end ? s : before, slot, wave);
                if (q > 0) {  // the products before these
                    const int g1 = (q - 1) >> 2, j1 = (q - 1) & 3;
#pragma unroll
                    for (int i = 0; i < GM; ++i) scale_add(acc[g1 * GM + i][j1], p[(q - 1) & 1][i], t[g1 & 1][i], f.fc, j1);
                }
                // in turn one product and the multiply-adds of the one GM before it
#pragma unroll
                for (int i = 0; i < GM; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, WIDE ? 4 : 1, 0);
                    if (end) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    else if (j == 0) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                    if (i == 0 && slot_ops(slot) == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                    if (i == 0 && slot_ops(slot) == 2) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
                    if (i == 0 && slot_ops(slot) >= 3) __builtin_amdgcn_sched_group_barrier(0x020, 3, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, BROW ? 8 : 4, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < GM; ++i) scale_add(acc[FM - GM + i][3], p[1][i], t[(NG - 1) & 1][i], f.fc, 3);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) pin(acc[i][j]);
        read_scales(f.fc, nx, l);
        f.st = sn;
    }

    // K-steps [k_lo, k_hi) of tile (m0, n0)
    __device__ __forceinline__ static void mainloop(f4 (&acc)[FM][4], const Fp8Args& a, lds_char* smem, int64_t m0, int64_t n0,
                                                    int k_lo, int k_hi, int wave, int lane) {
        const int wm = wave / WN, wn = wave % WN;
        Dma d;
        dma_setup(d, a, m0, n0, k_lo, k_hi, wave, lane);
        Lane l;
        {
            const int i = lane & 15, g = lane >> 4;
            const int ra = wm * TM + i, rb = wn * 64 + n_row(i);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                l.a[q] = ra * 128 + (((g + 4 * q) ^ swz_a(ra)) << 4);
                l.b[q] = A_BYTES + rb * 128 + (((g + 4 * q) ^ swz_b(rb)) << 4);
            }
            l.sa = SA_OFF + ra * 4;
            l.sb = SB_OFF + (wn * 64 + (BROW ? n_row(4 * g) : 0)) * 4;
        }
        // the step that needs mask_tail is the matrix's last
        const int last = (int)((a.K + 127) / 128) - 1, k_tail = (a.K & 15) && last < k_hi ? (int)(a.K & 127) : 0;
        // the first NST steps' copies: all of step 0 .. NST - 2, and of step NST - 1 what a K-step before it would have sent
#pragma unroll
        for (int i = 0; i < NST; ++i)
#pragma unroll
            for (int op = 0; op < (i < NST - 1 ? OPS : min(4 * PER_SLOT, OPS)); ++op) dma_op(d, smem + i * STAGE, op, wave);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * OPS + (4 * PER_SLOT < OPS ? 4 * PER_SLOT : OPS)) : "memory");
        barrier();
        if (k_tail && k_lo == last) mask_tail(smem, 0, k_tail, threadIdx.x);
        Pipe f;
        f.st = 0;
        read_rows(f.fr[0], smem, l, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) read_col(f.fc, smem, l, j);
        read_scales(f.fc, smem, l);
        int kt = k_lo;
        const int plain = k_tail && k_lo < last ? last - 1 : k_hi;
        for (; kt < plain; ++kt) kstep<false>(acc, f, d, l, smem, 0, wave);
        if (kt < k_hi) {
            kstep<true>(acc, f, d, l, smem, k_tail, wave);
            kstep<false>(acc, f, d, l, smem, 0, wave);
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // (nothing lands in LDS after the workgroup)
    }

    __device__ __forceinline__ static void run(const Fp8Args& a) {
        __shared__ __attribute__((aligned(1024))) char smem_raw[LDS];
        lds_char* smem = (lds_char*)smem_raw;
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int T = a.tiles_m * a.tiles_n;
        const int nidx = xcd_order(blockIdx.x, T * a.split);
        const int share = nidx / T, t = nidx - share * T;
        int tm, tn;
        super_order(t, a.tiles_m, a.tiles_n, a.group_m, a.super_m, a.super_n, &tm, &tn);
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        const int64_t steps = (a.K + 127) / 128;
        const int k_lo = (int)(share * steps / a.split), k_hi = (int)((share + 1) * steps / a.split);
        f4 acc[FM][4];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
        if (k_lo < k_hi) mainloop(acc, a, smem, m0, n0, k_lo, k_hi, wave, lane);
        if (a.split > 1) {
            f4* o = (f4*)a.ws + ((int64_t)nidx * NW + wave) * FM * 4 * 64 + lane;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[(i * 4 + j) * 64] = acc[i][j];
            return;
        }
        store_tile(acc, a, m0 + wm * TM + (lane & 15), n0 + wn * 64 + n_row(4 * (lane >> 4)));
    }
    // accumulators to C: row m of row tile 0, column n of tile 0
    __device__ __forceinline__ static void store_tile(const f4 (&acc)[FM][4], const Fp8Args& a, int64_t m, int64_t n) {
        constexpr int E = WIDE ? 4 : 16;  // consecutive columns a lane has
#pragma unroll
        for (int q = 0; q < 16 / E; ++q) {
            const int64_t nq = n + n_tile(q);
            if (nq >= a.N) continue;
            const Epilogue<E> epi(a, nq);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (m + 16 * i >= a.M) continue;
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = acc[i][(q * E + e) >> 2][e & 3];
                epi.store(v, m + 16 * i);
            }
        }
    }

    // Sum of a split launch (of either width): a wave takes one accumulator tile (16 rows by four columns a lane) and has up to eight
    // shares' partials of it in flight (one after the other, eleven shares of 37 rows took 6.3 us); they are added in
    // order.
    __device__ __forceinline__ static void run_sum(const Fp8Args& a) {
        const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
        const int64_t T = (int64_t)a.tiles_m * a.tiles_n;
        int64_t b = blockIdx.x;
        const int i = (int)(b % FM);
        b /= FM;
        const int wave = (int)(b % NW);
        const int t = (int)(b / NW);
        int tm, tn;
        super_order(t, a.tiles_m, a.tiles_n, a.group_m, a.super_m, a.super_n, &tm, &tn);
        const int wm = wave / WN, wn = wave % WN;
        const int64_t m = (int64_t)tm * BM + wm * TM + 16 * i + (lane & 15), n = (int64_t)tn * BN + wn * 64 + (a.c_type == C_ACC ? 4 * (lane >> 4) + 16 * j : 16 * (lane >> 4) + 4 * j);
        if (m >= a.M || n >= a.N) return;
        const f4* p = (const f4*)a.ws + ((((int64_t)t * NW + wave) * FM + i) * 4 + j) * 64 + lane;
        const int64_t step = T * NW * FM * 4 * 64;
        f4 s = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < a.split; k += 8) {
            f4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < a.split) x[u] = p[(k + u) * step];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < a.split) s += x[u];
        }
        const Epilogue<4> epi(a, n);
        float v[4] = {s[0], s[1], s[2], s[3]};
        epi.store(v, m);
    }
};

template <int CFG, bool A5, bool B5, bool BROW, bool WIDE>
__global__ __launch_bounds__((Tile<CFG, A5, B5, BROW, WIDE>::NT)) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_tile_kernel(Fp8Args a) {
    Tile<CFG, A5, B5, BROW, WIDE>::run(a);
}

template <int CFG, bool A5, bool B5, bool WIDE>
void launch_width(const Fp8Args& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n * a.split)), block(Tile<CFG, A5, B5, false, WIDE>::NT);
    if (a.b_row) hipLaunchKernelGGL((fp8_tile_kernel<CFG, A5, B5, true, WIDE>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((fp8_tile_kernel<CFG, A5, B5, false, WIDE>), grid, block, 0, s, a);
}
template <int CFG, bool A5, bool B5>
int launch_cfg(const Fp8Args& a, hipStream_t s) {
    if constexpr (kFp8Tiles[CFG].wide) {
        if (a.c_type == C_ACC) launch_width<CFG, A5, B5, true>(a, s);
        else launch_width<CFG, A5, B5, false>(a, s);
    } else {
        if (a.c_type == C_ACC) return -1;
        launch_width<CFG, A5, B5, false>(a, s);
    }
    return (int)hipGetLastError();
}
template <bool A5, bool B5>
int launch_types(int cfg, const Fp8Args& a, hipStream_t s) {
    static_assert(kNumFp8Tiles == 4, "one case a config");
    switch (cfg) {
    case 0: return launch_cfg<0, A5, B5>(a, s);
    case 1: return launch_cfg<1, A5, B5>(a, s);
    case 2: return launch_cfg<2, A5, B5>(a, s);
    default: return launch_cfg<3, A5, B5>(a, s);
    }
}

}  // namespace fp8t
}  // namespace tcm
