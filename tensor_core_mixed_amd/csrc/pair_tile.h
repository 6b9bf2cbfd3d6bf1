// Main loop of the tiled products whose 128-byte K-step is two 16-byte
// chunks a lane and row:
//
//   FP4    256 4-bit values of a row, a chunk one block of 32 with its scale:
//          two 16x16x128 matrix instructions a step, which take a block's
//          scale as an exponent and add the scaled blocks in binary32;
//   split  32 values of a row as two binary16 parts (the value is upper +
//          lower), upper parts in the first 64 bytes, lower ones in the
//          others: three 16x16x32 instructions a step, upper upper, upper
//          lower and lower upper.
//
// Both operands are rows with k contiguous, A [M][..], B [N][..].  The matrix
// instruction takes its first operand from B's rows and its second from A's,
// so a lane's accumulators run along n at one m and a row's stores are
// contiguous: row i of a wave's tiles j = 0 .. 3 is column 16 (i / 4) + 4 j +
// i % 4 of its 64 (16 columns a lane), or with WIDE 16 j + i (four columns a
// lane, four lanes side by side: binary32 C).
//
// Copies: 128-byte rows of each operand go to LDS by 16-byte direct loads,
// the chunk's place XOR-ed with a function of the row so that the reads of a
// fragment fall on distinct banks; NST stages, copies NST - 1 steps ahead, a
// few at a time between the products.  A lane takes the chunks 2g and 2g + 1
// of a row (g = lane / 16; FP4), so its two scales are neighbouring bytes of
// a word, one read; they lie at places g and g + 4.  Scale words travel with
// their step (4-byte direct loads, so that their rows need no alignment).
#pragma once
#include <hip/hip_runtime.h>

#include "lowp.h"
#include "tcm_internal.h"

namespace tcm {
namespace pair {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_void;

constexpr unsigned kOOB = 0x40000000u;  // past every descriptor's range: such loads give zeros
constexpr int kRsrcWord3 = 0x00020000;  // raw dword access

// What the main loop reads.  Rows at multiples of 16 bytes.
struct Operands {
    const unsigned char *A, *B;
    int64_t M, N, lda, ldb;   // rows, and bytes from one to the next
    int64_t row_bytes;        // of a row that hold values
    // FP4
    int64_t K;
    const unsigned *sa, *sb;  // [k / 128][row]
    int64_t ldsa, ldsb;
};

template <int BM_, int BN_, int WM_, int WN_, int NST_, bool FP4, bool WIDE>
struct Loop {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
    static constexpr int NW = WM * WN, NT = NW * 64;
    static constexpr int TM = BM / WM, FM = TM / 16;  // 16-row tiles of A a wave
    static_assert(BN / WN == 64, "a wave covers 64 columns");
    static constexpr int GM = FM >= 4 ? 2 : 1, NG = FM / GM;  // row tiles taken together, groups a K-step
    static_assert(FM % (2 * GM) == 0, "a step starts with the first of the two fragment buffers");
    static_assert(NW == 8 || NW == 4 || (NW == 2 && !FP4), "");
    static constexpr int NB = NW == 8 ? 1 : 8 / NW;  // offsets of B's copies: the swizzle of rows 8 NW apart differs
    static constexpr int IA = BM / (8 * NW), IB = BN / (8 * NW);
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + NW * 256;
    static constexpr int STAGE = FP4 ? SB_OFF + NW * 256 : SA_OFF;
    static constexpr int LDS = NST * STAGE;
    static_assert(LDS <= 160 * 1024 && (!FP4 || (2 * BM <= 64 * NW && 2 * BN <= 64 * NW)), "a wave copies 64 scale words of each operand");

    // The column of the wave's 64 that is row i of its tile j, and its parts: n_row(i) + n_tile(j).
    __device__ __forceinline__ static constexpr int n_row(int i) { return WIDE ? i : 16 * (i >> 2) + (i & 3); }
    __device__ __forceinline__ static constexpr int n_tile(int j) { return (WIDE ? 16 : 4) * j; }
    // Both swizzles of the row that a fragment read takes as its i-th are i / 2 % 8: any sixteen lanes that the LDS serves
    // at once then fall on distinct banks.
    __device__ __forceinline__ static int swz_a(int r) { return (r >> 1) & 7; }
    __device__ __forceinline__ static int swz_b(int r) { return WIDE ? (r >> 1) & 7 : ((r >> 1) & 1) | ((r >> 4) & 3) << 1; }
    // the chunk of a row that lies at place p before the swizzle
    __device__ __forceinline__ static int chunk(int p) { return FP4 ? (p & 3) << 1 | p >> 2 : p; }
    __device__ __forceinline__ static int place(int c) { return FP4 ? c >> 1 | (c & 1) << 2 : c; }

    // A wave's copies of a step: IA of A, IB of B, and one of each operand's scales.
    static constexpr int NS = FP4 ? 2 : 0, OPS = IA + IB + NS;
    struct Dma {
        unsigned a_off, b_off[NB], s_off[2];
        int a_k, b_k[NB], s_k[2];
        const unsigned char *pa, *pb;
        const unsigned* ps[2];
        int64_t s_step[2];  // words
        int s_lds[2];
        unsigned a_hop, b_hop;
        int a_range, b_range, k_left, steps_left;
        // of the step being copied: offsets, out of range past its data, and ranges, empty past the last step.  (The
        // range is checked against the lane's offset alone, so the whole of it goes there.)
        unsigned oa, ob[NB], os[2];
        int ra, rb;
    };
    __device__ __forceinline__ static void dma_setup(Dma& d, const Operands& a, int64_t m0, int64_t n0, int k_lo, int k_hi, int wave,
                                                     int lane) {
        {
            const int r = 8 * wave + (lane >> 3), c = chunk((lane & 7) ^ swz_a(r));
            d.a_off = (unsigned)(r * (int)a.lda + 16 * c);
            d.a_k = 16 * c;
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int r = 8 * (NW * q + wave) + (lane >> 3), c = chunk((lane & 7) ^ swz_b(r));
            d.b_off[q] = (unsigned)(r * (int)a.ldb + 16 * c);
            d.b_k[q] = 16 * c;
        }
        if constexpr (FP4) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // A's words, B's
                const int rows = q ? BN : BM;
                const int plane = 64 * wave / rows, i = 64 * wave % rows + lane;  // of the step's two words, and the row
                const int64_t r0 = q ? n0 : m0, ld = q ? a.ldsb : a.ldsa;
                d.s_off[q] = plane < 2 && r0 + i < (q ? a.N : a.M) ? (unsigned)(4 * i) : kOOB;
                d.s_k[q] = 64 * plane;
                d.ps[q] = (q ? a.sb : a.sa) + (2 * (int64_t)k_lo + (plane & 1)) * ld + r0;
                d.s_step[q] = 2 * ld;
                d.s_lds[q] = (q ? SB_OFF : SA_OFF) + wave * 256;
            }
        }
        const int64_t k0 = (int64_t)k_lo * 128;
        d.pa = a.A + m0 * a.lda + k0;
        d.pb = a.B + n0 * a.ldb + k0;
        d.a_hop = (unsigned)(8 * NW * (int)a.lda);
        d.b_hop = (unsigned)(8 * NW * NB * (int)a.ldb);
        // the ranges end with the last row's last 16-byte chunk (which may hold values past K)
        const int left = (int)(a.row_bytes - k0);
        const int rows_a = (int)min<int64_t>(a.M - m0, BM), rows_b = (int)min<int64_t>(a.N - n0, BN);
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
#pragma unroll
            for (int q = 0; q < NB; ++q) d.ob[q] = d.b_k[q] < left ? d.b_off[q] : kOOB;
#pragma unroll
            for (int q = 0; q < NS; ++q) d.os[q] = d.s_k[q] < left ? d.s_off[q] : kOOB;
        }
        if (op < IA) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(d.pa, d.ra), (lds_void*)(s + (NW * op + wave) * 1024), 16, d.oa + op * d.a_hop, 0, 0,
                                                     0);
        } else if (op < IA + IB) {
            const int j = op - IA;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(d.pb, d.rb), (lds_void*)(s + A_BYTES + (NW * j + wave) * 1024), 16,
                                                     d.ob[j % NB] + (j / NB) * d.b_hop, 0, 0, 0);
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

    // The last step of a K that does not fill it (FP4): zeros for A's values past K in the chunk that K ends in, and
    // for both operands' scale bytes of blocks past K, which may be NaN.  (Chunks past K are zeros already.)
    __device__ __forceinline__ static void mask_tail(lds_char* smem, int st, int krem, int tid) {
        const int c = krem >> 5, n = krem & 31, blocks = (krem + 31) >> 5;
        lds_char* s = smem + st * STAGE;
        for (int r = tid; r < BM + BN; r += NT) {
            if (r < BM && n) {
                __attribute__((address_space(3))) i4* p = (__attribute__((address_space(3))) i4*)(s + r * 128 + ((place(c) ^ swz_a(r)) << 4));
                i4 v = *p;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int k = n - 8 * d;
                    v[d] = k >= 8 ? v[d] : (k <= 0 ? 0 : (int)((unsigned)v[d] & (0xffffffffu >> (32 - 4 * k))));
                }
                *p = v;
            }
#pragma unroll
            for (int plane = 0; plane < 2; ++plane) {
                const int b = blocks - 4 * plane;
                __attribute__((address_space(3))) unsigned* w =
                    (__attribute__((address_space(3))) unsigned*)(s + (r < BM ? SA_OFF + (plane * BM + r) * 4 : SB_OFF + (plane * BN + r - BM) * 4));
                if (b < 4) *w = b <= 0 ? 0u : *w & (0xffffffffu >> (32 - 8 * b));
            }
        }
        __syncthreads();
    }

    struct Lane {
        int a[2], b[2];   // byte offsets within a stage of this lane's two chunks of row tile 0
        int sa, sb;
    };
    __device__ __forceinline__ static i4 read16(const lds_char* s, int o) { return *(const __attribute__((address_space(3))) i4*)(s + o); }
    __device__ __forceinline__ static int read_scales(const lds_char* s, int o) {
        return *(const __attribute__((address_space(3))) unsigned short*)(s + o);
    }

    struct Rows {  // a group of row tiles
        i4 a[GM][2];
        int s[GM];
    };
    struct Cols {
        i4 b[4][2];
        int s[4];
    };
    __device__ __forceinline__ static void read_rows(Rows& f, const lds_char* s, const Lane& l, int g) {
#pragma unroll
        for (int i = 0; i < GM; ++i) {
            f.a[i][0] = read16(s, l.a[0] + (g * GM + i) * 2048);
            f.a[i][1] = read16(s, l.a[1] + (g * GM + i) * 2048);
            if constexpr (FP4) f.s[i] = read_scales(s, l.sa + (g * GM + i) * 64);
        }
    }
    __device__ __forceinline__ static void read_col(Cols& f, const lds_char* s, const Lane& l, int j) {
        f.b[j][0] = read16(s, l.b[0] + n_tile(j) * 128);
        f.b[j][1] = read16(s, l.b[1] + n_tile(j) * 128);
        if constexpr (FP4) f.s[j] = read_scales(s, l.sb + n_tile(j) * 4);
    }
    __device__ __forceinline__ static i8v wide(i4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }
    // product Q of those that one accumulator takes in a step
    template <int Q>
    __device__ __forceinline__ static f4 mma(f4 acc, const Cols& b, int j, const Rows& a, int i) {
        if constexpr (FP4) {
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b.b[j][Q]), wide(a.a[i][Q]), acc, 4, 4, Q, b.s[j], Q, a.s[i]);
        } else {
            constexpr int x = Q == 1 ? 1 : 0, y = Q == 2 ? 1 : 0;  // (parts of B and of A)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, b.b[j][x]), __builtin_bit_cast(h8, a.a[i][y]), acc, 0, 0, 0);
        }
    }

    // (keeps the compiler from sinking products past the branches of the pipeline)
    __device__ __forceinline__ static void pin(f4& v) { asm volatile("" : "+v"(v)); }

    // The copies of step kt + NST go out a few at a time, from the last group of step kt (whose stage is then free) into
    // the groups of step kt + 1.  With two stages and two groups they have to land within the step: all at once.
    static constexpr int SLOTS = NG >= 4 ? 12 : (NST > 2 ? 8 : 4);
    static constexpr int PER_SLOT = (OPS + SLOTS - 1) / SLOTS;
    static constexpr int FIRST = 4 * PER_SLOT < OPS ? 4 * PER_SLOT : OPS;  // copies that a step sends in its last group
    __device__ __forceinline__ static void dma_slot(Dma& d, lds_char* s, int slot, int wave) {
#pragma unroll
        for (int i = 0; i < PER_SLOT; ++i)
            if (slot < SLOTS && slot * PER_SLOT + i < OPS) dma_op(d, s, slot * PER_SLOT + i, wave);
    }
    struct Pipe {
        Rows fr[2];
        Cols fc;
        int st;
    };
    // One K-step from stage f.st.  MASK: the next one is the matrix's last and K does not fill it.
    template <bool MASK>
    __device__ __forceinline__ static void kstep(f4 (&acc)[FM][4], Pipe& f, Dma& d, const Lane& l, lds_char* smem, int k_tail,
                                                 int wave) {
        lds_char* s = smem + f.st * STAGE;
        const int sn = f.st + 1 == NST ? 0 : f.st + 1;
        const lds_char* nx = smem + sn * STAGE;
        lds_char* before = smem + (f.st == 0 ? NST - 1 : f.st - 1) * STAGE;  // the stage of the step before
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            Rows& cur = f.fr[g & 1];
            Rows& nxt = f.fr[(g + 1) & 1];
            const bool end = g == NG - 1;
            __builtin_amdgcn_sched_barrier(0);  // (reads, copies and products stay within their group)
            if (!end) {
                read_rows(nxt, s, l, g + 1);
            } else {
                // every fragment of this step is in registers: the next step's copies must have landed, and those of
                // step kt + NST may overwrite this stage
                wait_copies<NST - 2>();
                barrier();
                if constexpr (MASK) mask_tail(smem, sn, k_tail, threadIdx.x);
                read_rows(nxt, nx, l, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = g * 4 + j, slot = end ? j : 4 + q;
#pragma unroll
                for (int i = 0; i < GM; ++i) acc[g * GM + i][j] = mma<0>(acc[g * GM + i][j], f.fc, j, cur, i);
#pragma unroll
                for (int i = 0; i < GM; ++i) acc[g * GM + i][j] = mma<1>(acc[g * GM + i][j], f.fc, j, cur, i);
                if constexpr (!FP4) {
#pragma unroll
                    for (int i = 0; i < GM; ++i) acc[g * GM + i][j] = mma<2>(acc[g * GM + i][j], f.fc, j, cur, i);
                }
                if (end) read_col(f.fc, nx, l, j);
                dma_slot(d, end ? s : before, slot, wave);
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) pin(acc[i][j]);
        f.st = sn;
    }

    // K-steps [k_lo, k_hi) of tile (m0, n0).  (split: `steps` of them, those from k_hi on with zeros, so that the parts of a
    // workgroup meet at as many barriers)
    __device__ __forceinline__ static void run(f4 (&acc)[FM][4], const Operands& a, lds_char* smem, int64_t m0, int64_t n0, int k_lo,
                                               int k_hi, int steps, int wave, int lane) {
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
            l.sa = SA_OFF + ((g >> 1) * BM + ra) * 4 + (g & 1) * 2;
            l.sb = SB_OFF + ((g >> 1) * BN + rb) * 4 + (g & 1) * 2;
        }
        // the step that needs mask_tail is the matrix's last
        const int last = (int)((a.row_bytes + 127) / 128) - 1, k_tail = FP4 && (a.K & 255) && last < k_hi ? (int)(a.K & 255) : 0;
        // the first NST steps' copies: all of step 0 .. NST - 2, and of step NST - 1 what a K-step before it would have sent
#pragma unroll
        for (int i = 0; i < NST; ++i)
#pragma unroll
            for (int op = 0; op < (i < NST - 1 ? OPS : FIRST); ++op) dma_op(d, smem + i * STAGE, op, wave);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * OPS + FIRST) : "memory");
        barrier();
        if (k_tail && k_lo == last) mask_tail(smem, 0, k_tail, threadIdx.x);
        Pipe f;
        f.st = 0;
        read_rows(f.fr[0], smem, l, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) read_col(f.fc, smem, l, j);
        if constexpr (FP4) {
            int kt = k_lo;
            const int plain = k_tail && k_lo < last ? last - 1 : k_hi;
            for (; kt < plain; ++kt) kstep<false>(acc, f, d, l, smem, 0, wave);
            if (kt < k_hi) {
                kstep<true>(acc, f, d, l, smem, k_tail, wave);
                kstep<false>(acc, f, d, l, smem, 0, wave);
            }
        } else {
            for (int i = 0; i < steps; ++i) kstep<false>(acc, f, d, l, smem, 0, wave);
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // (nothing lands in LDS after the workgroup)
    }
};

}  // namespace pair
}  // namespace tcm
