// Mixture-of-experts layer for a few tokens: over the pairs p = (token, slot)
// with expert e = ids[p],
//
//     h[p][i]   = weight[p] * silu(g) * u,   g, u = W1_gate[e], W1_up[e] row i . x[token],
//     y[p][c]   = W2[e] row c . h[p],
//     out[t][c] = sum over t's slots of y, in slot order.
//
// The chosen experts' weights bind the time.  A workgroup takes one expert
// and a block of its rows (16 of gate and up, 64 of W2) and multiplies them
// with all pairs of that expert, 16 (calls of up to 16 tokens) or 32 at a
// time, on 16x16x32 MFMAs with the weights' rows as one operand and the
// pairs as the other: weights are read once for every 16 or 32 pairs of their
// expert, and again in each part of kMoePairs pairs that a longer call is cut
// into.  They go straight from memory to registers; the waves deal k among
// themselves, the loads of the next steps in flight, and add their sums in LDS
// in wave order.  Every workgroup finds its pairs itself by one pass over the
// ids.  Three launches: up, down, sum over the slots.  (The sum left to the
// last workgroup of 64 columns took one token of eight experts from 17.9 to
// 17.3 us and four tokens from 47.5 to 48.6.)
//
// 24 bf16 tokens, four of 32 experts of 4096 x 1536 each, take 211 to 217 us,
// 5.4 TB/s, bound by memory, and in 8 bits 154 (3.7 TB/s: a step of an 8-bit
// row is half a line, and another wave reads the other half); one token of
// eight 8-bit experts of 2048 x 1024 18 us, of which 8 are its bytes.  2048
// tokens take 3.4 ms in bf16 and 2.7 in 8 bits (92 and 115 TFLOP/s): eight
// parts, each of which reads every expert once or twice.
//
// 8-bit weights are taken to 16-bit floats (exactly) and a 128-wide block's
// sums scaled by its tile's scale.  h goes to the matrix cores as the
// sum of two 16-bit parts: in bfloat16 a remainder of 2^-17; with float16
// weights it is binary32 in memory and taken to float16 after a power of two
// that brings the pair's largest |h| to 2^14 .. 2^15, 2^-22 of it or better.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace moe {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// Four waves a workgroup: with eight, a kernel past 128 registers leaves a CU one workgroup (24 bf16 tokens 243 us, 222
// with four, 237 with two; one token of eight 8-bit experts, of 4096 x 1536 46, 43 and 48, of 2048 x 1024 24, 22 and 27;
// 58 tokens of eleven 46 with eight and 37 with four).
constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kUpRows = 16;

// eight operand values of a lane, as raw bits of either 16-bit type
template <int XT>
__device__ __forceinline__ f4 mma(i4 w, i4 x, f4 c) {
    if constexpr (XT == F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, w), __builtin_bit_cast(f16x8_t, x), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w), __builtin_bit_cast(b8, x), c, 0, 0, 0);
}
template <int XT>
__device__ __forceinline__ i4 widen8(int w0, int w1) {
    if constexpr (XT == F16) {
        return __builtin_bit_cast(i4, fp8_to_f16x8<false>(w0, w1));
    } else {
        i4 r;
        r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, false));
        r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, true));
        r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, false));
        r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, true));
        return r;
    }
}

// 16 bytes at a 4-byte aligned address; load16_part: zeros past the row's `left` bytes
__device__ __forceinline__ i4 load16(const char* p) {
    i4 v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, 4), 16);
    return v;
}
__device__ __forceinline__ i4 load16_part(const char* p, int64_t left) {
    i4 v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // (rows are whole words; words past the row read its last)
        const int x = *(const int*)(p + min<int64_t>(4 * d, left - 4));
        v[d] = 4 * d < left ? x : 0;
    }
    return v;
}

// The pairs of this workgroup's expert in rising order: their number, with
// the expert in e.  Slot = an expert, or where there are fewer pairs than
// experts a pair, which serves its expert if it is the expert's first.
__device__ __forceinline__ int find_pairs(const MoeArgs& a, int slot, int* list, int* counts, int& e) {
    const int P = a.tokens * a.topk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool by_pair = P < a.experts;
    if (P <= 64) {
        // every wave by itself, from one load: all write the same list, and each reads what it wrote
        const int id = lane < P ? a.ids[lane] : -1;
        e = by_pair ? __builtin_amdgcn_readlane(id, slot) : slot;
        if ((unsigned)e >= (unsigned)a.experts) return 0;
        const unsigned long long m = __ballot(id == e);
        if (m == 0 || (by_pair && __builtin_ctzll(m) != slot)) return 0;
        if (id == e) list[__builtin_popcountll(m & ((1ull << lane) - 1))] = lane;
        __builtin_amdgcn_wave_barrier();
        return __builtin_popcountll(m);
    }
    e = by_pair ? a.ids[slot] : slot;
    if ((unsigned)e >= (unsigned)a.experts) return 0;
    int total = 0;
    for (int base = 0; base < P; base += kThreads) {
        const int p = base + tid;
        const bool hit = p < P && a.ids[p] == e;
        const unsigned long long m = __ballot(hit);
        __syncthreads();  // the counts of the pass before have been read
        if (lane == 0) counts[wave] = __builtin_popcountll(m);
        __syncthreads();
        int before = total;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += counts[w];
            total += counts[w];
        }
        if (hit) list[before + __builtin_popcountll(m & ((1ull << lane) - 1))] = p;
    }
    __syncthreads();
    if (by_pair && list[0] != slot) return 0;
    return total;
}

// ------------------------------------------------------------------- up

// A step is 64 k: of a weight row 16 bytes a lane (8-bit) or twice 16, k = 16 * (lane / 16) + ..
template <int XT, bool W8, int MT>
struct Up {
    static constexpr int WV = W8 ? 1 : 2;
    static constexpr int kAhead = MT == 1 ? 2 : 1;
    struct Step {
        i4 w[2][WV], x[MT][2];
        float s[2];
    };
    struct Src {
        const char *w[2], *x[MT];
        const float* s[2];
    };
    // step kt, whole or (PART) the row's last
    template <bool PART>
    __device__ __forceinline__ static void load(Step& t, const Src& s, const MoeArgs& a, int kt, int lane) {
        const int k = kt * 64 + 16 * (lane >> 4);
        constexpr int ES = W8 ? 1 : 2;
        if constexpr (!PART) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int v = 0; v < WV; ++v) t.w[m][v] = load16(s.w[m] + (int64_t)k * ES + 16 * v);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) t.x[i][v] = load16(s.x[i] + (int64_t)k * 2 + 16 * v);
        } else {
            const int64_t left = a.hidden - k;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int v = 0; v < WV; ++v) t.w[m][v] = load16_part(s.w[m] + (int64_t)k * ES + 16 * v, left * ES - 16 * v);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) t.x[i][v] = load16_part(s.x[i] + (int64_t)k * 2 + 16 * v, left * 2 - 16 * v);
        }
        if constexpr (W8) {
            t.s[0] = s.s[0][kt >> 1];
            t.s[1] = s.s[1][kt >> 1];
        }
    }
    __device__ __forceinline__ static void multiply(f4 (&acc)[2][MT], const Step& t) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            i4 w[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if constexpr (W8) w[v] = widen8<XT>(t.w[m][0][2 * v], t.w[m][0][2 * v + 1]);
                else w[v] = t.w[m][v];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if constexpr (W8) {
                    f4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < 2; ++v) p = mma<XT>(w[v], t.x[i][v], p);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[m][i][r] = __builtin_fmaf(p[r], t.s[m], acc[m][i][r]);
                } else {
#pragma unroll
                    for (int v = 0; v < 2; ++v) acc[m][i] = mma<XT>(w[v], t.x[i][v], acc[m][i]);
                }
            }
        }
    }
    // pairs list[0 .. n), n <= 16 MT
    __device__ __forceinline__ static void run(const MoeArgs& a, int e, int i0, const int* list, int n, f4* part) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int64_t mat = (int64_t)a.inter * a.hidden;
        const int row = min(i0 + (lane & 15), a.inter - 1);  // (rows past the matrix repeat the last: dropped)
        Src s;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            s.w[m] = (const char*)a.w1 + ((2 * (int64_t)e + m) * mat + (int64_t)row * a.hidden) * (W8 ? 1 : 2);
            if constexpr (W8)
                s.s[m] = a.s1 + ((2 * (int64_t)e + m) * scale_blocks(a.inter) + i0 / kScaleBlock) * scale_blocks(a.hidden);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
            s.x[i] = (const char*)a.x + (int64_t)(list[min(16 * i + (lane & 15), n - 1)] / a.topk) * a.ldx * 2;
        f4 acc[2][MT];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[m][i] = f4{0.f, 0.f, 0.f, 0.f};
        constexpr int OUT = (MT * 256 + kThreads - 1) / kThreads;  // results a thread
        float weight[OUT];
#pragma unroll
        for (int o = 0; o < OUT; ++o) weight[o] = a.weights[list[min((tid + o * kThreads) >> 4, n - 1)]];
        const int steps = a.hidden / 64;  // whole ones
        Step t[kAhead + 1];
        int kt = wave;
#pragma unroll
        for (int u = 0; u <= kAhead; ++u)
            if (kt + u * kWaves < steps) load<false>(t[u], s, a, kt + u * kWaves, lane);
        while (kt < steps) {
#pragma unroll
            for (int u = 0; u <= kAhead; ++u) {
                if (kt < steps) {
                    multiply(acc, t[u]);
                    if (kt + (kAhead + 1) * kWaves < steps) load<false>(t[u], s, a, kt + (kAhead + 1) * kWaves, lane);
                }
                kt += kWaves;
            }
        }
        if (a.hidden % 64 != 0 && wave == steps % kWaves) {
            load<true>(t[0], s, a, steps, lane);
            multiply(acc, t[0]);
        }
        __syncthreads();  // (part may still be read by a pass before)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < MT; ++i) part[((wave * 2 + m) * MT + i) * 64 + lane] = acc[m][i];
        __syncthreads();
#pragma unroll
        for (int o = 0; o < OUT; ++o) {
            const int x = tid + o * kThreads;
            if (x >= MT * 256) return;
            const int c = x >> 4, i = x & 15;  // pair of the pass, row of the block
            const float* q = (const float*)(part + (c >> 4) * 64 + (i >> 2) * 16 + (c & 15)) + (i & 3);
            float g = 0.f, u = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                g += q[(w * 2) * MT * 256];
                u += q[(w * 2 + 1) * MT * 256];
            }
            const bool live = c < n && i0 + i < a.inter;
            const int p = list[min(c, n - 1)];
            const float h = live ? weight[o] * (g / (1.f + expf(-g)) * u) : 0.f;
            if constexpr (XT == F16 && !W8) {
                if (live) ((float*)a.ws)[(int64_t)p * a.inter + i0 + i] = h;
            } else if (live) {  // both parts at once: the products would take them apart for every 64 rows of W2
                const __bf16 hi = (__bf16)h;
                const float rest = h - (float)hi;
                __bf16* o = (__bf16*)a.ws + 2 * (int64_t)p * a.inter + i0 + i;
                o[0] = hi;
                o[a.inter] = (__bf16)(rest == rest ? rest : 0.f);  // (an infinity has no remainder)
            }
            if constexpr (XT == F16 && !W8) {
                unsigned m = __builtin_bit_cast(unsigned, h) & 0x7fffffffu;
                for (int d = 8; d; d >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, d));
                if (i == 0 && c < n) a.hmax[(int64_t)p * ((a.inter + kUpRows - 1) / kUpRows) + i0 / kUpRows] = m;
            }
        }
    }
};

template <int XT, bool W8, int MT>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
    __shared__ f4 part[kWaves * 2 * MT * 64];
    __shared__ int list[kMoePairs], counts[kWaves];
    const int blocks = (a.inter + kUpRows - 1) / kUpRows;
    const int slot = blockIdx.x / blocks, i0 = (blockIdx.x % blocks) * kUpRows;
    int e;
    const int n = find_pairs(a, slot, list, counts, e);
    for (int j = 0; j < n; j += 16 * MT) {
        const int left = min(n - j, 16 * MT);
        if (left <= 16) Up<XT, W8, 1>::run(a, e, i0, list + j, left, part);
        else if constexpr (MT > 1) Up<XT, W8, MT>::run(a, e, i0, list + j, left, part);
    }
}

// ----------------------------------------------------------------- down

// float16 parts of eight values times f: v = hi + lo
__device__ __forceinline__ void split8(const i4 (&v)[2], float f, i4& hi, i4& lo) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const f4 q = __builtin_bit_cast(f4, v[d >> 1]);
        const float x = q[2 * (d & 1)] * f, y = q[2 * (d & 1) + 1] * f;
        const f16x2_t h = {(_Float16)x, (_Float16)y};
        const float dx = x - (float)h[0], dy = y - (float)h[1];
        const f16x2_t l = {(_Float16)(dx == dx ? dx : 0.f), (_Float16)(dy == dy ? dy : 0.f)};  // (infinities have no remainder)
        hi[d] = __builtin_bit_cast(int, h);
        lo[d] = __builtin_bit_cast(int, l);
    }
}

// Row tiles of W2 a workgroup (with two, 24 bf16 tokens of the layer above 217.0 us and 216.7 with four; one token of eight
// 8-bit experts 18.2 and 18.9).
constexpr int kDownTiles = 4, kDownRows = 16 * kDownTiles;

// A step is 32 k (8-bit weights: 64 k): 16 bytes of a row a lane.
template <int HT, bool W8, int MT>
struct Down {
    static constexpr int KV = W8 ? 2 : 1, KS = 32 * KV;
    static constexpr int kAhead = 1;
    struct Step {
        i4 w[kDownTiles];
        i4 h[MT][KV][2];  // eight k: binary32, or the two bfloat16 parts
        float s;
    };
    struct Src {
        const char* w[kDownTiles];
        const char* h[MT];
        const float* s;
    };
    // Chunk v of the step's h from k on, in the pair's 4 * inter bytes: four binary32 values, or eight of the row of upper
    // (v even) or lower parts; and the bytes left of it.
    __device__ __forceinline__ static int64_t h_offset(const MoeArgs& a, int k, int v) {
        return HT == F16 ? (int64_t)(k + 4 * v) * 4 : (int64_t)((v & 1) * (int64_t)a.inter + k + 8 * (v >> 1)) * 2;
    }
    __device__ __forceinline__ static int64_t h_left(int64_t left, int v) { return HT == F16 ? (left - 4 * v) * 4 : (left - 8 * (v >> 1)) * 2; }
    // step kt, whole or (PART) the row's last
    template <bool PART>
    __device__ __forceinline__ static void load(Step& t, const Src& s, const MoeArgs& a, int kt, int lane) {
        const int k = kt * KS + 8 * KV * (lane >> 4);
        constexpr int ES = W8 ? 1 : 2;
        if constexpr (!PART) {
#pragma unroll
            for (int j = 0; j < kDownTiles; ++j) t.w[j] = load16(s.w[j] + (int64_t)k * ES);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 2 * KV; ++v) t.h[i][v >> 1][v & 1] = load16(s.h[i] + h_offset(a, k, v));
        } else {
            const int64_t left = a.inter - k;
#pragma unroll
            for (int j = 0; j < kDownTiles; ++j) t.w[j] = load16_part(s.w[j] + (int64_t)k * ES, left * ES);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 2 * KV; ++v)
                    t.h[i][v >> 1][v & 1] = load16_part(s.h[i] + h_offset(a, k, v), h_left(left, v));
        }
        if constexpr (W8) t.s = s.s[kt >> 1];
    }
    __device__ __forceinline__ static void multiply(f4 (&acc)[kDownTiles][MT], const Step& t, const float (&f)[MT]) {
        i4 hi[MT][KV], lo[MT][KV];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                if constexpr (HT == F16) split8(t.h[i][v], f[i], hi[i][v], lo[i][v]);
                else hi[i][v] = t.h[i][v][0], lo[i][v] = t.h[i][v][1];
            }
#pragma unroll
        for (int j = 0; j < kDownTiles; ++j) {
            if constexpr (W8) {
                i4 w[KV];
#pragma unroll
                for (int v = 0; v < KV; ++v) w[v] = widen8<HT>(t.w[j][2 * v], t.w[j][2 * v + 1]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    f4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < KV; ++v) p = mma<HT>(w[v], hi[i][v], mma<HT>(w[v], lo[i][v], p));
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[j][i][r] = __builtin_fmaf(p[r], t.s, acc[j][i][r]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] = mma<HT>(t.w[j], hi[i][0], mma<HT>(t.w[j], lo[i][0], acc[j][i]));
            }
        }
    }
    __device__ __forceinline__ static void run(const MoeArgs& a, int e, int c0, const int* list, int n, f4* part, float* power) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int64_t mat = (int64_t)a.inter * a.hidden;
        constexpr bool kPower = HT == F16;
        float f[MT];
        if constexpr (kPower) {  // 2^e of every pair, e with |h| * 2^-e below 2^15
            const int nb = (a.inter + kUpRows - 1) / kUpRows;
            __syncthreads();
            for (int c = wave; c < n; c += kWaves) {
                unsigned m = 0;
                for (int b = lane; b < nb; b += 64) m = max(m, a.hmax[(int64_t)list[c] * nb + b]);
                for (int o = 32; o; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o));
                int x = (int)(m >> 23) - 127 - 14;
                if (m >= 0x7f800000u) x = 0;  // (infinities and NaN pass as they are)
                if (lane == 0) power[c] = __builtin_bit_cast(float, (unsigned)(max(x, -100) + 127) << 23);
            }
            __syncthreads();
        }
        Src s;
#pragma unroll
        for (int j = 0; j < kDownTiles; ++j) {
            const int row = min(c0 + 16 * j + (lane & 15), a.hidden - 1);
            s.w[j] = (const char*)a.w2 + ((int64_t)e * mat + (int64_t)row * a.inter) * (W8 ? 1 : 2);
        }
        if constexpr (W8) s.s = a.s2 + ((int64_t)e * scale_blocks(a.hidden) + c0 / kScaleBlock) * scale_blocks(a.inter);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int c = min(16 * i + (lane & 15), n - 1);
            s.h[i] = (const char*)a.ws + (int64_t)list[c] * a.inter * 4;
            f[i] = kPower ? 1.f / power[c] : 1.f;
        }
        f4 acc[kDownTiles][MT];
#pragma unroll
        for (int j = 0; j < kDownTiles; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = f4{0.f, 0.f, 0.f, 0.f};
        const int steps = a.inter / KS;  // whole ones
        Step t[kAhead + 1];
        int kt = wave;
#pragma unroll
        for (int u = 0; u <= kAhead; ++u)
            if (kt + u * kWaves < steps) load<false>(t[u], s, a, kt + u * kWaves, lane);
        while (kt < steps) {
#pragma unroll
            for (int u = 0; u <= kAhead; ++u) {
                if (kt < steps) {
                    multiply(acc, t[u], f);
                    if (kt + (kAhead + 1) * kWaves < steps) load<false>(t[u], s, a, kt + (kAhead + 1) * kWaves, lane);
                }
                kt += kWaves;
            }
        }
        if (a.inter % KS != 0 && wave == steps % kWaves) {
            load<true>(t[0], s, a, steps, lane);
            multiply(acc, t[0], f);
        }
        __syncthreads();  // (part may still be read by a pass before)
#pragma unroll
        for (int j = 0; j < kDownTiles; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) part[((wave * kDownTiles + j) * MT + i) * 64 + lane] = acc[j][i];
        __syncthreads();
        for (int x = tid; x < MT * 16 * kDownRows; x += kThreads) {
            const int c = x / kDownRows, r = x % kDownRows;  // pair of the pass, row of the block
            if (c >= n || c0 + r >= a.hidden) continue;
            const float* q = (const float*)(part + ((r >> 4) * MT + (c >> 4)) * 64 + ((r & 15) >> 2) * 16 + (c & 15)) + (r & 3);
            float y = q[0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) y += q[w * kDownTiles * MT * 256];
            if constexpr (kPower) y *= power[c];
            a.y[(int64_t)list[c] * a.hidden + c0 + r] = y;
        }
    }
};

template <int XT, bool W8, int MT>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
    constexpr int HT = W8 ? BF16 : XT;  // (8-bit weights are exact in either type)
    __shared__ f4 part[kWaves * kDownTiles * MT * 64];
    __shared__ float power[16 * MT];
    __shared__ int list[kMoePairs], counts[kWaves];
    const int blocks = (a.hidden + kDownRows - 1) / kDownRows;
    const int slot = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * kDownRows;
    int e;
    const int n = find_pairs(a, slot, list, counts, e);
    for (int j = 0; j < n; j += 16 * MT) {
        const int left = min(n - j, 16 * MT);
        if (left <= 16) Down<HT, W8, 1>::run(a, e, c0, list + j, left, part, power);
        else if constexpr (MT > 1) Down<HT, W8, MT>::run(a, e, c0, list + j, left, part, power);
    }
}

template <int XT>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = n / a.hidden;
    const int c = (int)(n - t * a.hidden);
    if (t >= a.tokens) return;
    float v = 0.f;
    for (int j = 0; j < a.topk; j += 8) {
        float y[8];  // (loads in flight together; a slot that adds nothing has no y)
        int e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t p = t * a.topk + min(j + u, a.topk - 1);
            e[u] = a.ids[p];
            y[u] = a.y[p * a.hidden + c];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j + u < a.topk && (unsigned)e[u] < (unsigned)a.experts) v += y[u];
    }
    store_c_any((char*)a.out + (t * a.ldo + c) * 2, XT == F16 ? C_F16 : C_BF16, v);
}

template <int XT, bool W8, int MT>
void launch_products(const MoeArgs& a, hipStream_t s) {
    const int slots = min(a.tokens * a.topk, a.experts);
    const dim3 up((unsigned)(slots * ((a.inter + kUpRows - 1) / kUpRows)));
    const dim3 down((unsigned)(slots * ((a.hidden + kDownRows - 1) / kDownRows)));
    hipLaunchKernelGGL((moe_up_kernel<XT, W8, MT>), up, dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL((moe_down_kernel<XT, W8, MT>), down, dim3(kThreads), 0, s, a);
}
template <int XT, bool W8>
int launch(const MoeArgs& a, hipStream_t s) {
    // an expert has a pair of every token at most (unless a token names it twice): 16 at a time, or up to 32
    if (a.tokens <= 16) launch_products<XT, W8, 1>(a, s);
    else launch_products<XT, W8, 2>(a, s);
    hipLaunchKernelGGL((moe_sum_kernel<XT>), dim3((unsigned)(((int64_t)a.tokens * a.hidden + 255) / 256)), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace moe

int launch_moe_tile(int x_type, bool w_e4m3, const MoeArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (x_type == F16) return w_e4m3 ? moe::launch<F16, true>(a, s) : moe::launch<F16, false>(a, s);
    return w_e4m3 ? moe::launch<BF16, true>(a, s) : moe::launch<BF16, false>(a, s);
}

}  // namespace tcm
