// What trains the router: how often each expert is chosen, the loss that
// balances them and the one that keeps the logits small, and the gradient of
// both, and of the chosen experts' weights, by the logits x.
//
//     p = softmax(x) over the experts, or s / (sum of s) with s = 1 / (1 + exp(-x)),
//     n_e = the choices of expert e, T = the tokens that count, k = topk,
//     balance = experts * sum_e (n_e / (T k)) * mean over tokens of p_e,
//     z = mean over tokens of log(sum_e exp(x_e))^2.
//
// With B = dL/dbalance * experts / (T^2 k), g_j = dL/dweight of slot j, G_e the
// sum of g over the slots that hold e, and w_j = s_j / (sum of the chosen s),
//
//     softmax:  dx_e = p_e B (n_e - sum n p)                          + z's
//                    + p_e scale (G_e - sum G p)                        (weights as they are)
//                    + scale * sum over slots j with e of w_j (g_j - sum g w)  (normalised)
//     sigmoid:  dx_e = (1 - s_e) p_e B (n_e - sum n p)                + z's
//                    + (1 - s_e) s_e scale G_e, or (1 - s_e) times the normalised sum,
//     z's = dL/dz * 2 log(sum exp x) / T * softmax(x)_e.
//
// The exponentials are binary32 ones; what is subtracted after them (G_e -
// sum G p loses all but 1 - p where one expert takes all) is formed in
// binary64 from them, where their relative errors stay relative errors.
//
// Sixteen lanes take a token of up to 256 experts, so a sum over them is four
// steps on the vector ALU for four tokens at once (a wave a token: gradient
// of 16384 x 256 28.5 us, now 12.8; losses' first launch 15.4, now 7.9); a wave
// takes one of more.  17.8 and 8.9 MB are not what bounds them: the vector ALU
// issues in 57% and 49% of the cycles (an exponential or two a value, the sums,
// binary64), with 1.9 waves a SIMD (231 and 136 registers; 256 workgroups of
// eight waves), which wait for their loads and row sums half of the time.  A lane
// holds runs of experts that one load brings.  The losses' sums run over a
// lane's tokens in registers, over a workgroup in LDS and over the workgroups
// in a second launch, each in a fixed order; counts are integers, whose order
// plays no part.  A lane adds the shares of 32 tokens at most in binary32 (they
// have one sign, so a long sum's roundings can all go one way: 2200 shares of
// 1 / 600 are off by 3e-5, 2^17 by 1.4e-3); those runs and what follows are
// added in binary64, with one rounding to binary32 a workgroup.  The longer
// calls have their own instance: 200000 x 384 168 to 170 us, where 16384 x 256
// would take 0.5 us more for what it does not need.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace balance {

typedef float f4_t __attribute__((ext_vector_type(4)));

// one step of a sum or a maximum over a row of 16 lanes: with the lane N places on.  (Every lane ends with the same
// bits: the two sides of a step add the same two numbers.)
template <int N>
__device__ __forceinline__ float ror(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, 0x120 + N, 0xf, 0xf, true);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), 0x120 + N, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <class V>
__device__ __forceinline__ V row_sum(V v) {
    v += ror<8>(v);
    v += ror<4>(v);
    v += ror<2>(v);
    return v + ror<1>(v);
}
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }  // (a NaN stays)
__device__ __forceinline__ float row_max(float v) {
    v = larger(v, ror<8>(v));
    v = larger(v, ror<4>(v));
    v = larger(v, ror<2>(v));
    return larger(v, ror<1>(v));
}
// over the lanes of a token
template <int LPT, class V>
__device__ __forceinline__ V token_sum(V v) {
    v = row_sum(v);
    if constexpr (LPT == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
    v = row_max(v);
    if constexpr (LPT == 64) {
        v = larger(v, __shfl_xor(v, 16));
        v = larger(v, __shfl_xor(v, 32));
    }
    return v;
}
// exp x for -104 <= x <= 80 to 2 steps of its last place: 2^t (1 + d ln 2), t + d = x log2 e with log2 e in two parts.
// (A NaN stays.)
__device__ __forceinline__ float exp_of(float x) {
    constexpr float hi = 0x1.715476p+0f, lo = 0x1.4ae0cp-26f, ln2 = 0x1.62e43p-1f;
    const float t = x * hi, d = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t)), r = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(r, d * ln2, r);
}
// and for any x <= 0
__device__ __forceinline__ float exp_neg(float x) { return exp_of(larger(x, -200.f)); }
// 1 / x to a step of its last place
__device__ __forceinline__ float inverse(float x) {
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.f), r, r);
}
__device__ __forceinline__ float log_of(float x) { return __builtin_amdgcn_logf(x) * 0x1.62e43p-1f; }
// (what an exponential takes: to 2^-23)
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.f) - log_of(1.f + exp_neg(-__builtin_fabsf(x))); }
// the sigmoid of x, and 1 minus it
__device__ __forceinline__ float sigmoid(float x, float* rest) {
    const float q = exp_neg(-__builtin_fabsf(x)), y = inverse(1.f + q), n = q * y;
    *rest = x >= 0.f ? n : y;
    return x >= 0.f ? y : (x < 0.f ? n : x);  // (a NaN stays)
}

constexpr float kPad = -120.f;  // its exponential is 0

// A token's experts over LPT lanes, NPL a lane, in runs of V: expert i of a lane is run i / V at V * lane.
template <int XT, int LPT, int NPL>
struct Layout {
    static constexpr int V = XT == F32 || NPL < 8 ? 4 : 8, RUN = V * LPT, ES = XT == F32 ? 4 : 2;
    __device__ __forceinline__ static int expert(int i, int sub) { return i / V * RUN + V * sub + i % V; }

    // Logits, kPad past the last expert.  True where a logit lies outside [-60, 40] or is a NaN.
    __device__ __forceinline__ static bool load(float (&x)[NPL], const void* base, int64_t t, int64_t ldx, int experts, int sub) {
        const char* row = (const char*)base + t * ldx * ES;
        float far = 0.f;
#pragma unroll
        for (int r = 0; r < NPL / V; ++r) {
            const int e = expert(r * V, sub);
            if (e + V <= experts) {
                unsigned w[V * ES / 4];
                __builtin_memcpy(w, row + (int64_t)e * ES, V * ES);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[r * V + i] = load_float<XT>((const char*)w, i);
                    far = larger(far, __builtin_fabsf(x[r * V + i] + 10.f));
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[r * V + i] = kPad;
                    if (e + i < experts) {
                        x[r * V + i] = load_float<XT>(row, e + i);
                        far = larger(far, __builtin_fabsf(x[r * V + i] + 10.f));
                    }
                }
            }
        }
        return !(far <= 50.f);
    }
    // kPad -> -inf
    __device__ __forceinline__ static void no_pad(float (&x)[NPL], int experts, int sub) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (expert(i, sub) >= experts) x[i] = -INFINITY;
    }
    __device__ __forceinline__ static void store(const float (&d)[NPL], const RouteGradArgs& a, int64_t t, int sub) {
        const int ds = c_elem_bytes(a.d_type);
        char* row = (char*)a.d + t * a.ldd * ds;
#pragma unroll
        for (int r = 0; r < NPL / V; ++r) {
            const int e = expert(r * V, sub);
            char* p = row + (int64_t)e * ds;
            if (e + V <= a.experts) {
                if (a.d_type == C_ACC) {
                    __builtin_memcpy(p, &d[r * V], 4 * V);
                } else {
                    unsigned w[V / 2];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float u = d[r * V + 2 * i], v = d[r * V + 2 * i + 1];
                        const unsigned lo = a.d_type == C_F16 ? __builtin_bit_cast(unsigned short, (_Float16)u) : __builtin_bit_cast(unsigned short, (__bf16)u);
                        const unsigned hi = a.d_type == C_F16 ? __builtin_bit_cast(unsigned short, (_Float16)v) : __builtin_bit_cast(unsigned short, (__bf16)v);
                        w[i] = lo | hi << 16;
                    }
                    __builtin_memcpy(p, w, 2 * V);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i < a.experts) store_c_any(p + i * ds, a.d_type, d[r * V + i]);
            }
        }
    }
};

// Of a token: exp(x - *at), and with SIG the sigmoids and 1 minus them.  False for a token of nothing but -inf.  Where
// every logit of a token lies near 0 (`far`: not), one exponential serves, and no maximum is needed.  A wave with a far
// token takes the long way for all, but by the same steps for the near ones, whose bits are the same anywhere.
template <int LPT, int NPL, class Y, bool SIG>
__device__ __forceinline__ bool scores(float (&e)[NPL], float (&s)[NPL], float (&r)[NPL], float* at, float (&x)[NPL], bool far, int experts,
                                       int sub) {
    if (!__ballot(far)) {
        *at = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            e[i] = exp_of(x[i]);
            if constexpr (SIG) {
                r[i] = inverse(1.f + e[i]);
                s[i] = e[i] * r[i];
            }
        }
        return true;
    }
    const bool near = LPT < 64 && !((__ballot(far) >> (threadIdx.x & 48)) & 0xffff);
    Y::no_pad(x, experts, sub);
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) mx = larger(mx, x[i]);
    mx = token_max<LPT>(mx);
    const bool live = near || !(mx == -INFINITY);
    *at = live && !near ? mx : 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        e[i] = exp_neg(x[i] - *at);
        if constexpr (SIG) {
            s[i] = sigmoid(x[i], &r[i]);
            const float y = inverse(1.f + e[i]);
            r[i] = near ? y : r[i];
            s[i] = near ? e[i] * y : s[i];
        }
    }
    return live;
}
// The sigmoids' ratios to the largest, where binary32 does not hold them well; their sum is `total`.
template <int LPT, int NPL, class Sum>
__device__ __forceinline__ void far_shares(float (&p)[NPL], Sum* total, const float (&x)[NPL], bool live, float at) {
    const bool mine = *total < (Sum)0x1p-100;
    if (!__ballot(live && mine)) return;
    const float top = log_sigmoid(at);
    Sum u = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const float y = x[i] == -INFINITY ? 0.f : exp_neg(log_sigmoid(x[i]) - top);
        p[i] = mine ? y : p[i];
        u += (Sum)p[i];
    }
    *total = token_sum<LPT>(u);
}

// (losses from sums: the choices' share of an expert is n_e / (T k); a +inf logit, whose sigmoid is 1, makes both NaN, as it
// does the softmax's)
__device__ __forceinline__ void store_losses(const BalanceArgs& a, double dot, double z, int valid) {
    const double t = valid > 0 ? valid : 1, k = a.topk > 0 ? a.topk : 1;
    a.losses[0] = z != z ? __builtin_nanf("") : (float)((double)a.experts * dot / (t * k * t));
    a.losses[1] = (float)(z / t);
}
__device__ __forceinline__ double wave_sum(double v) { return token_sum<64>(v); }
__device__ __forceinline__ int wave_sum(int v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// ONE: a single workgroup does everything.  Else it leaves its partial sums.  LONG: a lane takes more than kBalanceRun
// tokens, and adds the shares of so many to a binary64 sum.
template <int XT, int LPT, int NPL, bool SIG, bool ONE, bool LONG>
__global__ __launch_bounds__(64 * (ONE ? kBalanceOneWaves : kBalanceWaves)) void balance_kernel(BalanceArgs a) {
    using Y = Layout<XT, LPT, NPL>;
    constexpr int W = ONE ? kBalanceOneWaves : kBalanceWaves, E = NPL * LPT, TPW = 64 / LPT;
    __shared__ std::conditional_t<LONG, double, float> sp[W * TPW][E];
    __shared__ int hist[E], sv[W];
    __shared__ double sz[W], sd[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane % LPT, group = wave * TPW + lane / LPT;
    for (int e = tid; e < E; e += 64 * W) hist[e] = 0;
    __syncthreads();
    float acc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        acc[i] = 0.f;
        if constexpr (LONG) sp[group][Y::expert(i, sub)] = 0;
    }
    double z = 0;
    int valid = 0, run = 0;
    const int64_t step = (int64_t)gridDim.x * W * TPW;
    for (int64_t t0 = (int64_t)blockIdx.x * W * TPW; t0 < a.tokens; t0 += step) {
        if constexpr (LONG) {
            if (run++ == kBalanceRun) {
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    sp[group][Y::expert(i, sub)] += (double)acc[i];
                    acc[i] = 0.f;
                }
                run = 1;
            }
        }
        const int64_t t = t0 + group;
        const bool on = t < a.tokens && !(a.mask && a.mask[min(t, a.tokens - 1)] == 0);
        if (__ballot(on) == 0) continue;
        float x[NPL], e[NPL], p[NPL], r[NPL], at;
        bool far = false;
        if (on) {
            far = Y::load(x, a.x, t, a.ldx, a.experts, sub);
            for (int j = sub; j < a.topk; j += LPT) {
                const unsigned id = (unsigned)a.ids[t * a.topk + j];
                if (id < (unsigned)a.experts) atomicAdd(&hist[id], 1);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i) x[i] = 0.f;
        }
        const bool live = scores<LPT, NPL, Y, SIG>(e, p, r, &at, x, far, a.experts, sub) && on && a.experts > 0;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += e[i];
        sum = token_sum<LPT>(sum);
        float total = sum;
        if constexpr (SIG) {
            total = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) total += p[i];
            total = token_sum<LPT>(total);
            far_shares<LPT>(p, &total, x, live, at);
        }
        const float inv = live ? 1.f / total : 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] += live ? (SIG ? p[i] : e[i]) * inv : 0.f;
        if (sub == 0) {
            valid += on;
            const double lse = (double)at + (double)logf(sum);
            if (live) z += lse * lse;
        }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if constexpr (LONG) sp[group][Y::expert(i, sub)] += (double)acc[i];
        else sp[group][Y::expert(i, sub)] = acc[i];
    }
    z = wave_sum(z);
    valid = wave_sum(valid);
    if (lane == 0) sz[wave] = z, sv[wave] = valid;
    __syncthreads();
    z = 0, valid = 0;
    for (int w = 0; w < W; ++w) z += sz[w], valid += sv[w];
    double dot = 0;
    for (int e = tid; e < a.experts; e += 64 * W) {
        double s = 0;
#pragma unroll 8
        for (int g = 0; g < W * TPW; ++g) s += (double)sp[g][e];  // in the groups' order
        if constexpr (ONE) {
            a.counts[e] = hist[e];
            dot += (double)hist[e] * s;
        } else {
            a.p[(int64_t)blockIdx.x * a.experts + e] = (float)s;
            a.n[(int64_t)blockIdx.x * (a.experts + 1) + e] = hist[e];
        }
    }
    if constexpr (ONE) {
        dot = wave_sum(dot);
        if (lane == 0) sd[wave] = dot;
        __syncthreads();
        if (tid == 0) {
            dot = 0;
            for (int w = 0; w < W; ++w) dot += sd[w];
            a.counts[a.experts] = valid;
            store_losses(a, dot, z, valid);
        }
    } else if (tid == 0) {
        a.n[(int64_t)blockIdx.x * (a.experts + 1) + a.experts] = valid;
        a.z[blockIdx.x] = z;
        if (blockIdx.x == 0) *a.arrived = 0;  // (for the next launch)
    }
}

// The partial sums of 16 experts a workgroup (of 64: 8.4 us of 16384 x 256's, five of them reading on four CUs).  Their
// parts of sum n p / (T k T), which lies in [0, 1], are added as integers of 2^-49 in the word that also counts the
// arrivals (and those with a NaN, or anything else past 1): one atomic addition hands everything on, without a fence, and gives the same sum in
// any order.  (The loss is off by experts^2 / 16 * 2^-50 at most, 2^-34 for 1024 of them.)
constexpr int kJoinWaves = 16, kJoinExperts = 16, kJoinSlices = kJoinWaves * 4, kJoinRows = (kBalanceGroups + kJoinSlices - 1) / kJoinSlices;
constexpr int kFraction = 49, kNans = 50, kArrivals = 57;
static_assert((kRouteMaxExperts + kJoinExperts - 1) / kJoinExperts < 128, "counts of arrivals in 7 bits");
__global__ __launch_bounds__(64 * kJoinWaves) void balance_join_kernel(BalanceArgs a) {
    __shared__ double sp[kJoinWaves][kJoinExperts], sz[kBalanceGroups / 64];
    __shared__ int sn[kJoinWaves][kJoinExperts], sv[kBalanceGroups / 64];
    const int tid = threadIdx.x, lane = tid & 63, g = tid >> 6, e = blockIdx.x * kJoinExperts + (lane & 15);
    double p = 0, z = 0;
    int n = 0, valid = 0;
    if (tid < a.groups) z = a.z[tid], valid = a.n[(int64_t)tid * (a.experts + 1) + a.experts];
    if (e < a.experts) {
        float x[kJoinRows];  // (in flight together)
        int y[kJoinRows];
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            const int r = i * kJoinSlices + (tid >> 4);
            x[i] = r < a.groups ? a.p[(int64_t)r * a.experts + e] : 0.f;
            y[i] = r < a.groups ? a.n[(int64_t)r * (a.experts + 1) + e] : 0;
        }
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) p += (double)x[i], n += y[i];
    }
    p += __shfl_xor(p, 16);
    p += __shfl_xor(p, 32);
    n += __shfl_xor(n, 16);
    n += __shfl_xor(n, 32);
    if (lane < 16) sp[g][lane] = p, sn[g][lane] = n;
    if (tid < kBalanceGroups) {
        z = wave_sum(z);
        valid = wave_sum(valid);
        if (lane == 0) sz[g] = z, sv[g] = valid;
    }
    __syncthreads();
    if (tid >= 16) return;
    p = 0, n = 0;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i) p += sp[i][lane], n += sn[i][lane];
    if (e < a.experts) a.counts[e] = n;
    const double dot = row_sum((double)n * p);
    z = 0, valid = 0;
#pragma unroll
    for (int i = 0; i < kBalanceGroups / 64; ++i) z += sz[i], valid += sv[i];
    if (lane != 0) return;
    const double t = valid > 0 ? valid : 1, k = a.topk > 0 ? a.topk : 1, part = dot / (t * k * t);
    const uint64_t mine = part <= 1.5 ? (uint64_t)(part * (double)(1ull << kFraction) + 0.5) : 1ull << kNans;
    const uint64_t sum = mine + __hip_atomic_fetch_add(a.arrived, mine + (1ull << kArrivals), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((sum >> kArrivals) != gridDim.x - 1) return;
    const bool nan = ((sum >> kNans) & 127) || z != z;
    a.counts[a.experts] = valid;
    a.losses[0] = nan ? __builtin_nanf("") : (float)((double)a.experts * ((double)(sum & ((1ull << kNans) - 1)) / (double)(1ull << kFraction)));
    a.losses[1] = (float)(z / t);
}

template <int XT, int LPT, int NPL>
int balance_n(const BalanceArgs& a, hipStream_t s) {
    const auto launch = [&](auto sig, auto one, auto lng) {
        hipLaunchKernelGGL((balance_kernel<XT, LPT, NPL, sig(), one(), lng()>), dim3((unsigned)a.groups),
                           dim3(64 * (one() ? kBalanceOneWaves : kBalanceWaves)), 0, s, a);
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if (a.groups <= 1) {
        if (a.sigmoid) launch(yes, yes, no);
        else launch(no, yes, no);
    } else {
        const bool lng = a.tokens > (int64_t)a.groups * kBalanceWaves * (64 / LPT) * kBalanceRun;
        if (a.sigmoid) lng ? launch(yes, no, yes) : launch(yes, no, no);
        else lng ? launch(no, no, yes) : launch(no, no, no);
        hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)((a.experts + kJoinExperts - 1) / kJoinExperts)),
                           dim3(64 * kJoinWaves), 0, s, a);
    }
    return (int)hipGetLastError();
}

constexpr int kWaves = 4;

// SB: slots in blocks of 16, one a lane of a row (each row of a token holds them all)
template <int XT, int LPT, int NPL, int SB, bool SIG>
struct Grad {
    using Y = Layout<XT, LPT, NPL>;
    static constexpr int TPW = 64 / LPT;
    struct Slots {
        int id[SB];    // -1: none
        float v[SB];
    };
    static constexpr int E = LPT * NPL;
    __device__ __forceinline__ static void run(const RouteGradArgs& a) {
        __shared__ __attribute__((aligned(16))) float lds_g[kWaves * TPW][E];  // a token's G
        __shared__ __attribute__((aligned(16))) int lds_n[E];                  // counts
        const int tid = threadIdx.x, lane = tid & 63, sub = lane % LPT, slot = lane & 15, wave = tid >> 6;
        float* G = lds_g[wave * TPW + lane / LPT];
        // of the losses, the same for every token
        double bc = 0, zc = 0;
        if (a.dlosses) {
            const double t = a.counts[a.experts] > 0 ? a.counts[a.experts] : 1, k = a.topk > 0 ? a.topk : 1;
            bc = (double)a.dlosses[0] * a.experts / (t * t * k);
            zc = (double)a.dlosses[1] * 2 / t;
        }
        for (int e = tid; e < E; e += 64 * kWaves) lds_n[e] = a.dlosses && e < a.experts ? a.counts[e] : 0;
        __syncthreads();
        const auto count = [&](int i) { return (double)lds_n[Y::expert(i, sub)]; };
        const bool weights = a.dweights != nullptr;
        const double plain = a.norm ? 0.0 : (double)a.scale, normal = a.norm ? 1.0 : 0.0;  // what G counts for in the two forms of the weights
        const int64_t step = (int64_t)gridDim.x * kWaves * TPW;
        for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * TPW; t0 < a.tokens; t0 += step) {
            const int64_t t = t0 + lane / LPT, tt = min(t, a.tokens - 1);
            const bool on = t < a.tokens, masked = a.mask && a.mask[tt] == 0;
            float x[NPL], d[NPL];
            bool far = Y::load(x, a.x, tt, a.ldx, a.experts, sub);
            Slots s;
            float xs[SB];
#pragma unroll
            for (int b = 0; b < SB; ++b) {
                const int j = 16 * b + slot;
                s.id[b] = -1;
                s.v[b] = 0.f;
                xs[b] = -INFINITY;
                if (weights && j < a.topk) {
                    const int e = a.ids[tt * a.topk + j];
                    const float g = a.dweights[tt * a.topk + j];
                    if (!masked && (unsigned)e < (unsigned)a.experts) {
                        s.id[b] = e;
                        s.v[b] = g;
                        if (a.norm) xs[b] = load_float<XT>((const char*)a.x + tt * a.ldx * Y::ES, e);
                    }
                }
            }
            if (masked) {  // (whatever its logits hold)
                far = false;
#pragma unroll
                for (int i = 0; i < NPL; ++i) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < NPL; i += 4) *(f4_t*)(G + Y::expert(i, sub)) = f4_t{0.f, 0.f, 0.f, 0.f};
            // what a slot adds to its expert: to G, or (normalised weights) to the gradient itself
            if (weights && a.norm) {
                float top = -INFINITY, l[SB];
#pragma unroll
                for (int b = 0; b < SB; ++b) {
                    l[b] = a.sigmoid ? log_sigmoid(xs[b]) : xs[b];
                    if (s.id[b] < 0) l[b] = -INFINITY;
                    top = larger(top, l[b]);
                }
                top = row_max(top);
                double c[SB], n = 0, mean = 0;
#pragma unroll
                for (int b = 0; b < SB; ++b) {
                    c[b] = l[b] == -INFINITY ? 0.0 : (double)exp_neg(l[b] - top);
                    n += c[b];
                }
                n = row_sum(n);
                const double inv = n > 0 || n != n ? 1 / n : 0.0;
#pragma unroll
                for (int b = 0; b < SB; ++b) {
                    c[b] *= inv;
                    mean += (double)s.v[b] * c[b];
                }
                mean = row_sum(mean);
#pragma unroll
                for (int b = 0; b < SB; ++b) s.v[b] = (float)(c[b] * ((double)s.v[b] - mean) * a.scale);
            }
            if (weights) {
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
#pragma unroll
                for (int b = 0; b < SB; ++b)
                    if (s.id[b] >= 0 && sub < 16) atomicAdd(G + s.id[b], s.v[b]);  // (an id may repeat)
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
            }
            float soft[NPL], at;
            const auto g_of = [&](int i) { return (double)G[Y::expert(i, sub)]; };
            if constexpr (!SIG) {
                const bool live = scores<LPT, NPL, Y, false>(soft, x, x, &at, x, far, a.experts, sub) && !masked;
                double total = 0, dot = 0, dot_g = 0;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    total += (double)soft[i];
                    dot += (double)soft[i] * count(i);
                    dot_g += (double)soft[i] * g_of(i);
                }
                total = token_sum<LPT>(total);
                const double inv = 1 / total;
                dot = token_sum<LPT>(dot) * inv;
                dot_g = token_sum<LPT>(dot_g) * inv;
                const double zt = zc * ((double)at + (double)logf((float)total)) * inv, b = inv * bc, w = inv * plain;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const double g = g_of(i);
                    d[i] = (float)((double)soft[i] * (b * (count(i) - dot) + zt + w * (g - dot_g)) + normal * g);
                    if (!live) d[i] = 0.f;
                }
            } else {
                float sg[NPL], r[NPL];
                const bool live = scores<LPT, NPL, Y, true>(soft, sg, r, &at, x, far, a.experts, sub) && !masked;
                // (p, the shares, in d's place)
                double total = 0, st = 0, dot = 0;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    d[i] = sg[i];
                    total += (double)soft[i];
                    st += (double)d[i];
                }
                total = token_sum<LPT>(total);
                st = token_sum<LPT>(st);
                const double zt = zc * ((double)at + (double)logf((float)total)) / total;
                far_shares<LPT>(d, &st, x, live, at);
#pragma unroll
                for (int i = 0; i < NPL; ++i) dot += (double)d[i] * count(i);
                const double inv = 1 / st;
                dot = token_sum<LPT>(dot) * inv;
                const double b = inv * bc;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    d[i] = (float)((double)r[i] * ((double)d[i] * (b * (count(i) - dot)) + ((double)sg[i] * plain + normal) * g_of(i)) + zt * (double)soft[i]);
                    if (!live) d[i] = 0.f;
                }
            }
            if (on) Y::store(d, a, t, sub);
        }
    }
};

template <int XT, int LPT, int NPL, int SB, bool SIG>
__global__ __launch_bounds__(64 * kWaves) void route_grad_kernel(RouteGradArgs a) {
    Grad<XT, LPT, NPL, SB, SIG>::run(a);
}
template <int XT, int LPT, int NPL, int SB>
void launch_grad(const RouteGradArgs& a, dim3 grid, hipStream_t s) {
    if (a.sigmoid) hipLaunchKernelGGL((route_grad_kernel<XT, LPT, NPL, SB, true>), grid, dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((route_grad_kernel<XT, LPT, NPL, SB, false>), grid, dim3(64 * kWaves), 0, s, a);
}

template <int XT, int LPT, int NPL>
int grad_n(const RouteGradArgs& a, hipStream_t s) {
    constexpr int per = kWaves * 64 / LPT;
    const int64_t wgs = (a.tokens + per - 1) / per;
    const dim3 grid((unsigned)(wgs < 4096 ? wgs : 4096));
    if (a.topk <= 16) launch_grad<XT, LPT, NPL, 1>(a, grid, s);
    else launch_grad<XT, LPT, NPL, 4>(a, grid, s);
    return (int)hipGetLastError();
}

// the instance for so many experts
template <int XT, class F>
int for_experts(int experts, F f) {
    if (experts <= 64) return f.template operator()<XT, 16, 4>();
    if (experts <= 128) return f.template operator()<XT, 16, 8>();
    if (experts <= 256) return f.template operator()<XT, 16, 16>();
    if (experts <= 512) return f.template operator()<XT, 64, 8>();
    return f.template operator()<XT, 64, 16>();
}
template <class F>
int for_type(int x_type, int experts, F f) {
    switch (x_type) {
    case F16: return for_experts<F16>(experts, f);
    case BF16: return for_experts<BF16>(experts, f);
    default: return for_experts<F32>(experts, f);
    }
}
struct LaunchBalance {
    const BalanceArgs& a;
    hipStream_t s;
    template <int XT, int LPT, int NPL>
    int operator()() const { return balance_n<XT, LPT, NPL>(a, s); }
};
struct LaunchGrad {
    const RouteGradArgs& a;
    hipStream_t s;
    template <int XT, int LPT, int NPL>
    int operator()() const { return grad_n<XT, LPT, NPL>(a, s); }
};

}  // namespace balance

int launch_balance(int x_type, const BalanceArgs& a, void* stream) {
    return balance::for_type(x_type, a.experts, balance::LaunchBalance{a, (hipStream_t)stream});
}
int launch_route_grad(int x_type, const RouteGradArgs& a, void* stream) {
    return balance::for_type(x_type, a.experts, balance::LaunchGrad{a, (hipStream_t)stream});
}

}  // namespace tcm
