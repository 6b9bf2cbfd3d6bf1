// Expert router: the topk experts of every token by their logits and the
// weights of their outputs,
//
//     score = softmax(x) or 1 / (1 + exp(-x)),   key = score + bias, or x without a bias,
//     ids = the topk largest keys in falling order, ties to the lower expert,
//     weight = score[id] * scale, or with norm score[id] / (sum over ids of score) * scale.
//
// Both scores rise with x, so without a bias the logits order the experts
// exactly.  With a bias the keys count in binary64: near ones would change
// places in 32 bits.  Chosen scores of zero (a row of -inf) give weights of
// zero; a NaN key ranks above every number.
//
// One wave takes one token, expert e on lane e % 64.  Each pass takes the
// wave's largest remaining key, as order-preserving 32-bit integers, by a
// maximum over the lanes on the vector ALU, and the first expert that holds
// it; lane j keeps choice j and works out its weight at the end.  Keys with a
// bias are formed in binary32 first, off by less than half kSlack of the largest
// score and of the key: a token two of whose topk + 1 first keys lie closer
// than that is routed again by the binary64 passes, as is one with a NaN or a
// +inf or whose logits are all -inf, or with a chosen score under 2^-100, which
// binary32 holds in few bits or not at all (normalised weights are ratios, the
// same however small the scores are).  8192 tokens of 256 experts with a bias,
// eight chosen, take 10 us, bound by the instructions of the nine passes (25 us
// by binary64 passes alone).
#include <hip/hip_runtime.h>

#include <cmath>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace route {

constexpr int kWaves = 4;

// unsigned integers in the order of the floats, -0 with +0, every NaN on top
__device__ __forceinline__ uint64_t ordered(double v) {
    if (v != v) return ~0ull;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ unsigned ordered(float v) {  // (v is no NaN)
    const unsigned b = __builtin_bit_cast(unsigned, v + 0.f);
    return (b >> 31) ? ~b : b | (1u << 31);
}
__device__ __forceinline__ float unordered(unsigned k) { return __builtin_bit_cast(float, (k >> 31) ? k & 0x7fffffffu : ~k); }

template <int CTRL>
__device__ __forceinline__ unsigned max_step(unsigned v) {
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
    return v > o ? v : o;
}
// the largest over the wave, uniform: rows of 16 (shifts by 1, 2, 4, 8), then their last lanes handed on
__device__ __forceinline__ unsigned wave_max(unsigned v) {
    v = max_step<0x118>(max_step<0x114>(max_step<0x112>(max_step<0x111>(v))));
    v = max_step<0x143>(max_step<0x142>(v));
    return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL>
__device__ __forceinline__ float add_step(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = add_step<0x118>(add_step<0x114>(add_step<0x112>(add_step<0x111>(v))));
    v = add_step<0x143>(add_step<0x142>(v));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Twice the error of a binary32 key, as a share of the largest score and of
// |key|.  Of the score: the exponential's argument (|x| e^-|x| / ln 2 steps of
// 2^-24 at most, under 1), its value, the sum (NPL + 5 additions in softmax),
// the quotient and the product come to NPL + 11 steps of 2^-24; of the key:
// the bias's addition, one.
template <int NPL>
constexpr float kSlack = NPL > 4 ? 0x1p-18f : 0x1p-19f;

// One token in binary32; false where the binary64 passes have to take it.
template <int XT, int NPL, bool BIAS>
__device__ __forceinline__ bool route_fast(const RouteArgs& a, int64_t t, int lane) {
    const char* row = (const char*)a.x + t * a.ldx * (XT == F32 ? 4 : 2);
    float x[NPL];
    unsigned key[NPL];
    float mx = -INFINITY;
    bool odd = false;  // a NaN
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < a.experts ? load_float<XT>(row, e) : -INFINITY;
        odd |= x[i] != x[i];
        mx = x[i] > mx ? x[i] : mx;
    }
    if (__ballot(odd)) return false;
    mx = unordered(wave_max(ordered(mx)));
    if (!(mx > -INFINITY && mx < INFINITY)) return false;
    float sum = 0.f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += __expf(x[i] - mx);
        sum = wave_sum(sum);
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        float k = x[i];
        if constexpr (BIAS) {
            const float s = a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-x[i])) : __expf(x[i] - mx) * inv;
            k = s + (e < a.experts ? load_float<F32>((const char*)a.bias, e) : 0.f);
            odd |= !(k > -INFINITY && k < INFINITY);
        }
        key[i] = e < a.experts ? ordered(k) : 0;
    }
    if constexpr (BIAS) {
        if (__ballot(odd)) return false;
    }
    const float slack = a.sigmoid ? kSlack<NPL> : kSlack<NPL> * inv;  // (of the largest score)
    const int passes = BIAS ? min(a.topk + 1, a.experts) : a.topk;
    int my_id = 0;
    float my_x = 0.f, last = INFINITY;
    for (int j = 0; j < passes; ++j) {
        unsigned m = key[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) m = key[i] > m ? key[i] : m;
        m = wave_max(m);
        if constexpr (BIAS) {
            const float k = unordered(m);
            if (last - k <= slack + kSlack<NPL> * (k < 0.f ? -k : k)) return false;
            last = k;
        }
        bool found = false;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (found) continue;
            const unsigned long long h = __ballot(key[i] == m);
            if (h == 0) continue;
            found = true;
            const int l = __builtin_ctzll(h);
            if (lane == l) key[i] = 0;
            const float xv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x[i]), l));
            if (lane == j) my_id = i * 64 + l, my_x = xv;
        }
    }
    float w = 0.f;
    if (lane < a.topk) w = a.sigmoid ? 1.f / (1.f + expf(-my_x)) : expf(my_x - mx) * inv;
    if (__ballot(lane < a.topk && w < 0x1p-100f && my_x > -INFINITY)) return false;
    if (a.norm) {
        const float total = wave_sum(w);
        w = total == 0.f ? 0.f : w / total;
    }
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = my_id;
        a.weights[t * a.topk + lane] = w * a.scale;
    }
    return true;
}

template <int XT, int NPL, bool BIAS>
__device__ __forceinline__ void route_exact(const RouteArgs& a, int64_t t, int lane) {
    const char* row = (const char*)a.x + t * a.ldx * (XT == F32 ? 4 : 2);
    double sc[NPL];  // this lane's scores
    uint64_t key[NPL];
    float x[NPL];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < a.experts ? load_float<XT>(row, e) : -INFINITY;
        mx = (x[i] > mx || x[i] != x[i]) ? x[i] : mx;  // (a NaN stays)
    }
    double sum = 0;
    if (!a.sigmoid) {
        for (int o = 32; o; o >>= 1) {
            const float y = __shfl_xor(mx, o);
            mx = (y > mx || y != y) ? y : mx;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            sc[i] = mx == -INFINITY ? 0.0 : exp((double)x[i] - (double)mx);
            sum += i * 64 + lane < a.experts ? sc[i] : 0.0;
        }
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < NPL; ++i) sc[i] = sum == 0 ? 0.0 : sc[i] / sum;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) sc[i] = 1.0 / (1.0 + exp(-(double)x[i]));
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        key[i] = e >= a.experts ? 0 : ordered(BIAS ? sc[i] + (double)load_float<F32>((const char*)a.bias, e) : (double)x[i]);
    }
    int my_id = 0;  // lane j keeps choice j
    double my_score = 0, total = 0;
    for (int j = 0; j < a.topk; ++j) {
        // the largest upper half, then among its holders the largest lower half
        unsigned hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) hi = max(hi, (unsigned)(key[i] >> 32));
        hi = wave_max(hi);
#pragma unroll
        for (int i = 0; i < NPL; ++i) lo = (unsigned)(key[i] >> 32) == hi ? max(lo, (unsigned)key[i]) : lo;
        lo = wave_max(lo);
        const uint64_t m = (uint64_t)hi << 32 | lo;
        bool found = false;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (found) continue;
            const unsigned long long h = __ballot(key[i] == m);
            if (h == 0) continue;
            found = true;
            const int l = __builtin_ctzll(h);
            if (lane == l) key[i] = 0;
            const double s = __shfl(sc[i], l);
            if (lane == j) my_id = i * 64 + l, my_score = s;
            total += s;
        }
    }
    double w = my_score;
    if (a.norm) {
        w /= total;
        if (total < 0x1p-900) {
            // near the end of binary64's range or past it: differences of log-scores (up to a constant) keep the ratios
            double ls = lane < a.topk ? (double)load_float<XT>(row, my_id) : -INFINITY;
            if (a.sigmoid) ls = fmin(ls, 0.0) - log1p(exp(-fabs(ls)));
            double top = ls;
            for (int o = 32; o; o >>= 1) top = fmax(top, __shfl_xor(top, o));
            w = top == -INFINITY ? 0.0 : exp(ls - top);
            total = w;
            for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
            w = top == -INFINITY ? 0.0 : w / total;
        }
    }
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = my_id;
        a.weights[t * a.topk + lane] = (float)(w * (double)a.scale);
    }
}

template <int XT, int NPL, bool BIAS>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
    if (!route_fast<XT, NPL, BIAS>(a, t, lane)) route_exact<XT, NPL, BIAS>(a, t, lane);
}

template <int XT, int NPL>
int launch_n(const RouteArgs& a, hipStream_t s) {
    const int64_t per = (int64_t)kWaves << 23;  // tokens per launch, which counts its threads in 32 bits
    for (int64_t t = 0; t < a.tokens; t += per) {
        RouteArgs e = a;
        e.tokens = a.tokens - t < per ? a.tokens - t : per;
        e.x = (const char*)a.x + t * a.ldx * (XT == F32 ? 4 : 2);
        e.ids = a.ids + t * a.topk;
        e.weights = a.weights + t * a.topk;
        const dim3 grid((unsigned)((e.tokens + kWaves - 1) / kWaves));
        if (a.bias) hipLaunchKernelGGL((route_kernel<XT, NPL, true>), grid, dim3(64 * kWaves), 0, s, e);
        else hipLaunchKernelGGL((route_kernel<XT, NPL, false>), grid, dim3(64 * kWaves), 0, s, e);
    }
    return (int)hipGetLastError();
}
template <int XT>
int launch_x(const RouteArgs& a, hipStream_t s) {
    if (a.experts <= 64) return launch_n<XT, 1>(a, s);
    if (a.experts <= 128) return launch_n<XT, 2>(a, s);
    if (a.experts <= 256) return launch_n<XT, 4>(a, s);
    if (a.experts <= 512) return launch_n<XT, 8>(a, s);
    return launch_n<XT, 16>(a, s);
}

}  // namespace route

int launch_route(int x_type, const RouteArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (x_type) {
    case F16: return route::launch_x<F16>(a, s);
    case BF16: return route::launch_x<BF16>(a, s);
    default: return route::launch_x<F32>(a, s);
    }
}

}  // namespace tcm
