// Expert router: the topk experts of every token by their logits and the
// weights of their outputs,
//
//     score = softmax(x) or 1 / (1 + exp(-x)),   key = score + bias, or x without a bias,
//     ids = the topk largest keys in falling order, ties to the lower expert,
//     weight = score[id] * scale, or with norm score[id] / (sum over ids of score) * scale.
//
// Both scores rise with x, so without a bias the logits order the experts
// exactly.  With a bias the keys are formed in binary64: near ones would
// change places in 32 bits.  A sum of zero (a row of -inf) gives weights of
// zero; a NaN key ranks above every number.
//
// One wave takes one token, expert e on lane e % 64; the topk passes each
// take the wave's largest remaining key, compared as order-preserving
// integers.
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

template <int XT, int NPL, bool BIAS>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
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
    int my_id = 0;       // lane j keeps choice j
    double my_score = 0, total = 0;
    unsigned taken = 0;  // of this lane's values
    for (int j = 0; j < a.topk; ++j) {
        uint64_t best = 0;
        int be = 1 << 30;
        double bs = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 64 + lane;
            if (e < a.experts && !((taken >> i) & 1) && (be == 1 << 30 || key[i] > best)) best = key[i], be = e, bs = sc[i];
        }
        for (int o = 32; o; o >>= 1) {
            const uint64_t ok = __shfl_xor(best, o);
            const int oe = __shfl_xor(be, o);
            const double os = __shfl_xor(bs, o);
            if (oe != 1 << 30 && (be == 1 << 30 || ok > best || (ok == best && oe < be))) best = ok, be = oe, bs = os;
        }
        if ((be & 63) == lane) taken |= 1u << (be >> 6);
        if (j == lane) my_id = be, my_score = bs;
        total += bs;
    }
    if (lane < a.topk) {
        double w = my_score;
        if (a.norm) w = total == 0 ? 0.0 : w / total;
        a.ids[t * a.topk + lane] = my_id;
        a.weights[t * a.topk + lane] = (float)(w * (double)a.scale);
    }
}

template <int XT, int NPL>
int launch_n(const RouteArgs& a, hipStream_t s) {
    const int64_t per = (int64_t)kWaves << 30;  // tokens per launch
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
