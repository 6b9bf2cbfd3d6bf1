// Mixture-of-experts layer for any alignment and size: over the pairs
// p = (token, slot) with expert e = ids[p],
//
//     h[p][i]   = weight[p] * silu(g) * u,   g, u = W1_gate[e], W1_up[e] row i . x[token],
//     out[t][c] = sum over t's slots of W2[e] row c . h[p],
//
// one wave per dot product, two launches; h in binary32.  A pair whose id
// lies outside [0, experts) adds nothing.
#include <hip/hip_runtime.h>

#include "fp8_util.h"
#include "lowp.h"

namespace tcm {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ float wave_sum(float v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// element (r, c) of a rows x cols weight matrix, its tile scale applied
template <int XT, bool W8>
__device__ __forceinline__ float weight_at(const char* w, const float* s, int r, int c, int cols) {
    if constexpr (W8)
        return fp8_decode<false>(((const unsigned char*)w)[(int64_t)r * cols + c]) *
               load_float<F32>((const char*)s, (int64_t)(r / kScaleBlock) * scale_blocks(cols) + c / kScaleBlock);
    else return load_float<XT>(w, (int64_t)r * cols + c);
}

template <int XT, bool W8>
__global__ __launch_bounds__(64 * kWaves) void moe_up_generic(MoeArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int64_t p = n / a.inter;
    const int i = (int)(n - p * a.inter);
    if (p >= (int64_t)a.tokens * a.topk) return;
    const int64_t e = a.ids[p];
    float g = 0.f, u = 0.f;
    if (e >= 0 && e < a.experts) {
        const int64_t mat = (int64_t)a.inter * a.hidden, sm = scale_blocks(a.inter) * scale_blocks(a.hidden);
        const char* wg = (const char*)a.w1 + 2 * e * mat * (W8 ? 1 : 2);
        const char* wu = wg + mat * (W8 ? 1 : 2);
        const float* sg = W8 ? a.s1 + 2 * e * sm : nullptr;
        const char* x = (const char*)a.x + p / a.topk * a.ldx * 2;
        for (int k = lane; k < a.hidden; k += 64) {
            const float xv = load_float<XT>(x, k);
            g = __builtin_fmaf(weight_at<XT, W8>(wg, sg, i, k, a.hidden), xv, g);
            u = __builtin_fmaf(weight_at<XT, W8>(wu, W8 ? sg + sm : nullptr, i, k, a.hidden), xv, u);
        }
    }
    g = wave_sum(g);
    u = wave_sum(u);
    if (lane == 0) ((float*)a.ws)[p * a.inter + i] = a.weights[p] * (g / (1.f + expf(-g)) * u);
}

template <int XT, bool W8>
__global__ __launch_bounds__(64 * kWaves) void moe_down_generic(MoeArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int64_t t = n / a.hidden;
    const int c = (int)(n - t * a.hidden);
    if (t >= a.tokens) return;
    float y = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        const int64_t p = t * a.topk + j;
        const int64_t e = a.ids[p];
        if (e < 0 || e >= a.experts) continue;
        const int64_t mat = (int64_t)a.inter * a.hidden, sm = scale_blocks(a.inter) * scale_blocks(a.hidden);
        const char* w = (const char*)a.w2 + e * mat * (W8 ? 1 : 2);
        const float* s = W8 ? a.s2 + e * sm : nullptr;
        const float* h = (const float*)a.ws + p * a.inter;
        for (int i = lane; i < a.inter; i += 64) y = __builtin_fmaf(weight_at<XT, W8>(w, s, c, i, a.inter), h[i], y);
    }
    y = wave_sum(y);
    if (lane == 0) store_c_any((char*)a.out + (t * a.ldo + c) * 2, XT == F16 ? C_F16 : C_BF16, y);
}

template <int XT, bool W8>
int launch(const MoeArgs& a, hipStream_t s) {
    const int64_t up = (int64_t)a.tokens * a.topk * a.inter, down = (int64_t)a.tokens * a.hidden;
    if (up > 0)  // (without slots the outputs are zeros)
        hipLaunchKernelGGL((moe_up_generic<XT, W8>), dim3((unsigned)((up + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, s, a);
    hipLaunchKernelGGL((moe_down_generic<XT, W8>), dim3((unsigned)((down + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace

int launch_moe_generic(int x_type, bool w_e4m3, const MoeArgs& a, void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (x_type == F16) return w_e4m3 ? launch<F16, true>(a, s) : launch<F16, false>(a, s);
    return w_e4m3 ? launch<BF16, true>(a, s) : launch<BF16, false>(a, s);
}

}  // namespace tcm
