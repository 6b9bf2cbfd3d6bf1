// What trains the router: how often each expert is chosen, the loss that
// balances them and the one that keeps the logits small, and the gradient of
// both, and of the chosen experts' weights, by the logits x.
//
//     p = softmax(x) over the experts, or s / (sum of s) with s = 1 / (1 + exp(-x)),
//     n_e = the choices of expert e, T = the tokens that count, k = topk,
//     balance = experts * sum_e (n_e / (T k)) * mean over tokens of p_e,
//     z = mean over tokens of log(sum_e exp(x_e))^2.
//
// With u_e = B n_e (B = dL/dbalance * experts / (T^2 k)), G_e the sum of
// dL/dweight over the slots that hold e, and w_j = s_j / (sum of the chosen s),
//
//     softmax:  dx_e = p_e (u_e - sum u p)                          + z's
//                    + p_e scale (G_e - sum G p)                      (weights as they are)
//                    + scale * sum over slots j with e of w_j (g_j - sum g w)  (normalised)
//     sigmoid:  dx_e = (1 - s_e) p_e (u_e - sum u p)                + z's
//                    + (1 - s_e) s_e scale G_e, or (1 - s_e) times the normalised sum,
//     z's = dL/dz * 2 log(sum exp x) / T * softmax(x)_e.
//
// The exponentials are binary32 ones; what is subtracted after them (G_e -
// sum G p loses all but 1 - p where one expert takes all) is formed in
// binary64 from them, where their relative errors stay relative errors.
//
// One wave takes one token, expert e on lane e % 64.  The losses' sums run
// over a wave's tokens in registers, over a workgroup's waves in LDS and over
// the workgroups in a second launch, each in a fixed order; counts are
// integers, whose order plays no part.
#include <hip/hip_runtime.h>

#include <cmath>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace balance {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// with -inf (as no lane's neighbour) where a row of 16 ends
template <int CTRL>
__device__ __forceinline__ float max_step(float v) {
    const int none = (int)0xff800000u;
    const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(none, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    return __builtin_elementwise_maximum(v, o);  // (a NaN stays)
}
__device__ __forceinline__ float last_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
    v = max_step<0x118>(max_step<0x114>(max_step<0x112>(max_step<0x111>(v))));
    return last_lane(max_step<0x143>(max_step<0x142>(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0x111>(v);
    v += dpp<0x112>(v);
    v += dpp<0x114>(v);
    v += dpp<0x118>(v);
    v += dpp<0x142>(v);
    return last_lane(v + dpp<0x143>(v));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, 0xf, 0xf, false);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0x111>(v);
    v += dpp<0x112>(v);
    v += dpp<0x114>(v);
    v += dpp<0x118>(v);
    v += dpp<0x142>(v);
    v += dpp<0x143>(v);
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)b, 63), hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.f) - log1pf(expf(-__builtin_fabsf(x))); }

template <int XT, int NPL>
__device__ __forceinline__ void load_row(float (&x)[NPL], const void* base, int64_t t, int64_t ldx, int experts, int lane) {
    const char* row = (const char*)base + t * ldx * (XT == F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < experts ? load_float<XT>(row, e) : -INFINITY;
    }
}

// The scores' shares p of a token, up to the factor 1 / *total, and the log of the sum of exp x.  False for a token of
// nothing but -inf, whose shares are zero.
template <int NPL>
__device__ __forceinline__ bool shares(float (&p)[NPL], float* total, float* lse, const float (&x)[NPL], bool sigmoid, int lane) {
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) mx = __builtin_elementwise_maximum(mx, x[i]);
    mx = wave_max(mx);
    if (mx == -INFINITY) return false;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        p[i] = expf(x[i] - mx);
        s += p[i];
    }
    s = wave_sum(s);
    *lse = mx + logf(s);
    if (sigmoid) {
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            p[i] = 1.f / (1.f + expf(-x[i]));
            u += p[i];
        }
        s = wave_sum(u);
        if (s < 0x1p-100f) {  // (ratios to the largest keep their bits)
            const float top = log_sigmoid(mx);
            u = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                p[i] = x[i] == -INFINITY ? 0.f : expf(log_sigmoid(x[i]) - top);
                u += p[i];
            }
            s = wave_sum(u);
        }
    }
    *total = s;
    return true;
}

// Sums of tokens first, first + step, ..: this lane's experts' shares in acc, the others in LDS or returned.
template <int XT, int NPL>
__device__ __forceinline__ void sum_tokens(float (&acc)[NPL], double* z, int* valid, int* hist, const BalanceArgs& a, int64_t first,
                                           int64_t step, int lane) {
    for (int64_t t = first; t < a.tokens; t += step) {
        if (a.mask && a.mask[t] == 0) continue;
        ++*valid;
        for (int j = lane; j < a.topk; j += 64) {
            const unsigned id = (unsigned)a.ids[t * a.topk + j];
            if (id < (unsigned)a.experts) atomicAdd(&hist[id], 1);
        }
        float x[NPL], p[NPL], total, lse;
        load_row<XT, NPL>(x, a.x, t, a.ldx, a.experts, lane);
        if (!shares(p, &total, &lse, x, a.sigmoid, lane)) continue;
        const float inv = 1.f / total;
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] += p[i] * inv;
        *z += (double)lse * (double)lse;
    }
}

// (losses from sums: the choices' share of an expert is n_e / (T k))
__device__ __forceinline__ void store_losses(const BalanceArgs& a, double dot, double z, int valid) {
    const double t = valid > 0 ? valid : 1, k = a.topk > 0 ? a.topk : 1;
    a.losses[0] = (float)((double)a.experts * dot / (t * k * t));
    a.losses[1] = (float)(z / t);
}

// ONE: a single workgroup does everything.  Else it leaves its partial sums.
template <int XT, int NPL, bool ONE>
__global__ __launch_bounds__(64 * (ONE ? kBalanceOneWaves : kBalanceWaves)) void balance_kernel(BalanceArgs a) {
    constexpr int W = ONE ? kBalanceOneWaves : kBalanceWaves, E = NPL * 64;
    __shared__ float sp[E];
    __shared__ int hist[E], sv[W];
    __shared__ double sz[W], sd[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < E; e += 64 * W) hist[e] = 0, sp[e] = 0.f;
    __syncthreads();
    float acc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) acc[i] = 0.f;
    double z = 0;
    int valid = 0;
    sum_tokens<XT, NPL>(acc, &z, &valid, hist, a, (int64_t)blockIdx.x * W + wave, (int64_t)gridDim.x * W, lane);
    if (lane == 0) sz[wave] = z, sv[wave] = valid;
    for (int w = 0; w < W; ++w) {  // in the waves' order
        if (wave == w) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) sp[i * 64 + lane] += acc[i];
        }
        __syncthreads();
    }
    z = 0, valid = 0;
    for (int w = 0; w < W; ++w) z += sz[w], valid += sv[w];
    if constexpr (ONE) {
        double dot = 0;
        for (int e = tid; e < a.experts; e += 64 * W) {
            a.counts[e] = hist[e];
            dot += (double)hist[e] * (double)sp[e];
        }
        dot = wave_sum(dot);
        if (lane == 0) sd[wave] = dot;
        __syncthreads();
        if (tid == 0) {
            dot = 0;
            for (int w = 0; w < W; ++w) dot += sd[w];
            a.counts[a.experts] = valid;
            store_losses(a, dot, z, valid);
        }
    } else {
        float* p = a.p + (int64_t)blockIdx.x * a.experts;
        int* n = a.n + (int64_t)blockIdx.x * (a.experts + 1);
        for (int e = tid; e < a.experts; e += 64 * W) p[e] = sp[e], n[e] = hist[e];
        if (tid == 0) {
            n[a.experts] = valid;
            a.z[blockIdx.x] = z;
            if (blockIdx.x == 0) *a.arrived = 0;  // (for the next launch)
        }
    }
}

// The partial sums of 64 experts a workgroup; the last to arrive adds the workgroups' parts in order.
constexpr int kJoin = 16;
__global__ __launch_bounds__(64 * kJoin) void balance_join_kernel(BalanceArgs a) {
    __shared__ double sp[kJoin][64];
    __shared__ int sn[kJoin][64];
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
    double p = 0;
    int n = 0;
    if (e < a.experts) {
#pragma unroll 4
        for (int r = g; r < a.groups; r += kJoin) {
            p += (double)a.p[(int64_t)r * a.experts + e];
            n += a.n[(int64_t)r * (a.experts + 1) + e];
        }
    }
    sp[g][lane] = p;
    sn[g][lane] = n;
    __syncthreads();
    if (g != 0) return;
    p = 0, n = 0;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) p += sp[i][lane], n += sn[i][lane];
    if (e < a.experts) a.counts[e] = n;
    const double dot = wave_sum((double)n * p);
    int arrived = 0;
    if (lane == 0) {
        __hip_atomic_store(&a.share[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        arrived = __hip_atomic_fetch_add(a.arrived, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__shfl(arrived, 0) != (int)gridDim.x - 1) return;
    double z = 0;
    int valid = 0;
    for (int r = lane; r < a.groups; r += 64) {
        z += a.z[r];
        valid += a.n[(int64_t)r * (a.experts + 1) + a.experts];
    }
    z = wave_sum(z);
    for (int o = 32; o; o >>= 1) valid += __shfl_xor(valid, o);
    if (lane == 0) {
        double sum = 0;
        for (unsigned b = 0; b < gridDim.x; ++b) sum += __hip_atomic_load(&a.share[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        a.counts[a.experts] = valid;
        store_losses(a, sum, z, valid);
    }
}

template <int XT, int NPL>
int balance_n(const BalanceArgs& a, hipStream_t s) {
    if (a.groups <= 1) {
        hipLaunchKernelGGL((balance_kernel<XT, NPL, true>), dim3(1), dim3(64 * kBalanceOneWaves), 0, s, a);
    } else {
        hipLaunchKernelGGL((balance_kernel<XT, NPL, false>), dim3((unsigned)a.groups), dim3(64 * kBalanceWaves), 0, s, a);
        hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)((a.experts + 63) / 64)), dim3(64 * kJoin), 0, s, a);
    }
    return (int)hipGetLastError();
}

constexpr int kWaves = 4;

template <int XT, int NPL>
__device__ __forceinline__ void store_row(const float (&d)[NPL], const RouteGradArgs& a, int64_t t, int lane) {
    char* row = (char*)a.d + t * a.ldd * c_elem_bytes(a.d_type);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        if (e < a.experts) store_c_any(row + e * c_elem_bytes(a.d_type), a.d_type, d[i]);
    }
}

template <int XT, int NPL>
__global__ __launch_bounds__(64 * kWaves) void route_grad_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 63;
    // of the losses, the same for every token
    int count[NPL];
    double bc = 0, zc = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) count[i] = 0;
    if (a.dlosses) {
        const double t = a.counts[a.experts] > 0 ? a.counts[a.experts] : 1, k = a.topk > 0 ? a.topk : 1;
        bc = (double)a.dlosses[0] * a.experts / (t * t * k);
        zc = (double)a.dlosses[1] * 2 / t;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 64 + lane;
            if (e < a.experts) count[i] = a.counts[e];
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
        float d[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) d[i] = 0.f;
        float x[NPL], mx = -INFINITY;
        load_row<XT, NPL>(x, a.x, t, a.ldx, a.experts, lane);
#pragma unroll
        for (int i = 0; i < NPL; ++i) mx = i ? __builtin_elementwise_maximum(mx, x[i]) : x[i];
        mx = wave_max(mx);
        if ((a.mask && a.mask[t] == 0) || mx == -INFINITY) {
            store_row<XT, NPL>(d, a, t, lane);
            continue;
        }
        // this lane's slot
        int id = -1;
        float g = 0.f, xs = -INFINITY;
        if (a.dweights && lane < a.topk) {
            const int j = a.ids[t * a.topk + lane];
            if ((unsigned)j < (unsigned)a.experts) {
                id = j;
                g = a.dweights[t * a.topk + lane];
                xs = load_float<XT>((const char*)a.x + t * a.ldx * (XT == F32 ? 4 : 2), j);
            }
        }
        // what it adds to its expert: to G, or (normalised weights) to the gradient itself
        if (a.dweights && a.norm) {
            const float l = a.sigmoid ? log_sigmoid(xs) : xs, top = wave_max(id < 0 ? -INFINITY : l);
            const double c = id < 0 || l == -INFINITY ? 0.0 : (double)expf(l - top), n = wave_sum(c);
            const double w = n > 0 || n != n ? c / n : 0.0, mean = wave_sum((double)g * w);
            g = (float)(w * ((double)g - mean) * a.scale);
        }
        float G[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) G[i] = 0.f;
        if (a.dweights) {
            for (int j = 0; j < a.topk; ++j) {
                const int e = __builtin_amdgcn_readlane(id, j);
                const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), j));
                if (e < 0) continue;
#pragma unroll
                for (int i = 0; i < NPL; ++i) G[i] += i * 64 + lane == e ? v : 0.f;
            }
        }
        double p[NPL], total = 0, dot = 0, dot_g = 0;
        float soft[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            soft[i] = expf(x[i] - mx);
            total += (double)soft[i];
        }
        total = wave_sum(total);
        const double zt = zc == 0 ? 0 : zc * ((double)mx + (double)logf((float)total)) / total;
        const bool plain = a.dweights && !a.norm;
        if (!a.sigmoid) {
            const double inv = 1 / total;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                p[i] = (double)soft[i] * inv;
                dot += p[i] * (double)count[i];
                dot_g += p[i] * (double)G[i];
            }
            dot = wave_sum(dot);
            if (plain) dot_g = wave_sum(dot_g);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const double g = plain ? p[i] * ((double)G[i] - dot_g) * a.scale : (double)G[i];
                d[i] = (float)(p[i] * bc * ((double)count[i] - dot) + g + zt * (double)soft[i]);
            }
        } else {
            float s[NPL], r[NPL];  // the sigmoid and 1 minus it
            double st = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const float q = expf(-__builtin_fabsf(x[i])), y = 1.f / (1.f + q), n = q * y;
                s[i] = x[i] >= 0.f ? y : n;
                r[i] = x[i] >= 0.f ? n : y;
                if (x[i] != x[i]) s[i] = r[i] = x[i];
                p[i] = (double)s[i];
                st += p[i];
            }
            st = wave_sum(st);
            if (st < 0x1p-100) {  // (ratios to the largest keep their bits)
                const float top = log_sigmoid(mx);
                st = 0;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    p[i] = x[i] == -INFINITY ? 0.0 : (double)expf(log_sigmoid(x[i]) - top);
                    st += p[i];
                }
                st = wave_sum(st);
            }
            const double inv = 1 / st;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                p[i] *= inv;
                dot += p[i] * (double)count[i];
            }
            dot = wave_sum(dot);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const double g = plain ? (double)s[i] * (double)G[i] * a.scale : (double)G[i];
                d[i] = (float)((double)r[i] * (p[i] * bc * ((double)count[i] - dot) + g) + zt * (double)soft[i]);
            }
        }
        store_row<XT, NPL>(d, a, t, lane);
    }
}

template <int XT, int NPL>
int grad_n(const RouteGradArgs& a, hipStream_t s) {
    const int64_t wgs = (a.tokens + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((route_grad_kernel<XT, NPL>), dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(64 * kWaves), 0, s, a);
    return (int)hipGetLastError();
}

// the instance for so many experts
template <int XT, class F>
int for_experts(int experts, F f) {
    if (experts <= 64) return f.template operator()<XT, 1>();
    if (experts <= 128) return f.template operator()<XT, 2>();
    if (experts <= 256) return f.template operator()<XT, 4>();
    if (experts <= 512) return f.template operator()<XT, 8>();
    return f.template operator()<XT, 16>();
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
    template <int XT, int NPL>
    int operator()() const { return balance_n<XT, NPL>(a, s); }
};
struct LaunchGrad {
    const RouteGradArgs& a;
    hipStream_t s;
    template <int XT, int NPL>
    int operator()() const { return grad_n<XT, NPL>(a, s); }
};

}  // namespace balance

int launch_balance(int x_type, const BalanceArgs& a, void* stream) {
    return balance::for_type(x_type, a.experts, balance::LaunchBalance{a, (hipStream_t)stream});
}
int launch_route_grad(int x_type, const RouteGradArgs& a, void* stream) {
    return balance::for_type(x_type, a.experts, balance::LaunchGrad{a, (hipStream_t)stream});
}

}  // namespace tcm
