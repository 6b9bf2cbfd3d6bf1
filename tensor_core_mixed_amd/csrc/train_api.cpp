// C ABI of the router's losses and gradient (declared in include/tcm.h):
// argument checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "api_util.h"
#include "lowp.h"
#include "tcm_internal.h"

namespace tcm {
namespace {

int balance_impl(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, const int* ids,
                 const uint8_t* mask, int* counts, float* losses, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    if (t != F16 && t != BF16 && t != F32) return TCM_ERR_INVALID_VALUE;
    if (flags & ~TCM_ROUTE_SIGMOID) return TCM_ERR_INVALID_VALUE;
    if (tokens < 0 || experts < 0 || topk < 0 || tokens >= kDim || topk > experts) return TCM_ERR_INVALID_VALUE;
    if (ldx < std::max<int64_t>(experts, 1)) return TCM_ERR_INVALID_VALUE;
    if (experts > kRouteMaxExperts || topk > kRouteMaxTopk) return TCM_ERR_NOT_SUPPORTED;
    if (tokens * topk >= kDim) return TCM_ERR_NOT_SUPPORTED;  // (counts are 32-bit)
    if (!counts || !losses || (tokens > 0 && ((experts > 0 && !logits) || (topk > 0 && !ids)))) return TCM_ERR_INVALID_VALUE;
    if (!word_aligned(ids) || !word_aligned(counts) || !word_aligned(losses)) return TCM_ERR_INVALID_VALUE;
    const int64_t xb = span_of(tokens, experts, ldx, elem_bytes(t));
    if (xb < 0) return TCM_ERR_INVALID_VALUE;
    const Region out[2] = {{counts, (experts + 1) * 4}, {losses, 8}}, in[3] = {{logits, xb}, {ids, tokens * topk * 4}, {mask, tokens}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    BalanceArgs a{};
    a.x = logits;
    a.tokens = tokens;
    a.ldx = ldx;
    a.experts = (int)experts;
    a.topk = (int)topk;
    a.sigmoid = (flags & TCM_ROUTE_SIGMOID) != 0;
    a.ids = ids;
    a.mask = mask;
    a.counts = counts;
    a.losses = losses;
    a.groups = tokens <= kBalanceOneTokens || experts == 0
                   ? 1
                   : (int)std::min<int64_t>(kBalanceGroups, (tokens + kBalanceWaves - 1) / kBalanceWaves);
    std::unique_lock<std::mutex> order;
    if (a.groups > 1) {
        const int64_t joins = (experts + 63) / 64, g = a.groups;
        void* ws = nullptr;
        const int st = workspace_for(stream, 8 * g + 8 * joins + 4 * g * experts + 4 * g * (experts + 1) + 4, &ws, &order);
        if (st != TCM_OK) return st;
        a.z = (double*)ws;
        a.share = a.z + g;
        a.p = (float*)(a.share + joins);
        a.n = (int*)(a.p + g * experts);
        a.arrived = a.n + g * (experts + 1);
    }
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=balance tokens=%lld experts=%lld topk=%lld dtype=%d groups=%d%s%s", (long long)v[0], (long long)v[1],
                     (long long)v[2], (int)v[3], (int)v[4], v[5] ? " sigmoid=1" : "", v[6] ? " mask=1" : "");
        },
        {tokens, experts, topk, t, a.groups, a.sigmoid, mask != nullptr});
    return done(launch_balance(t, a, stream));
}

int route_grad_impl(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, float scale,
                    const int* ids, const uint8_t* mask, const float* dweights, const int* counts, const float* dlosses, void* D,
                    int64_t ldd, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    if (t != F16 && t != BF16 && t != F32) return TCM_ERR_INVALID_VALUE;
    if (flags & ~(TCM_ROUTE_SIGMOID | TCM_ROUTE_NORM | TCM_C_F16 | TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if ((flags & TCM_C_F16) && (flags & TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if (tokens < 0 || experts < 0 || topk < 0 || tokens >= kDim || topk > experts) return TCM_ERR_INVALID_VALUE;
    if (ldx < std::max<int64_t>(experts, 1) || ldd < std::max<int64_t>(experts, 1)) return TCM_ERR_INVALID_VALUE;
    if (experts > kRouteMaxExperts || topk > kRouteMaxTopk) return TCM_ERR_NOT_SUPPORTED;
    if (tokens == 0 || experts == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!logits || !D || (dweights && topk > 0 && !ids) || (dlosses && !counts)) return TCM_ERR_INVALID_VALUE;
    if (!word_aligned(ids) || !word_aligned(dweights) || !word_aligned(counts) || !word_aligned(dlosses)) return TCM_ERR_INVALID_VALUE;
    const int d_type = (flags & TCM_C_F16) ? C_F16 : ((flags & TCM_C_BF16) ? C_BF16 : C_ACC);
    const int64_t xb = span_of(tokens, experts, ldx, elem_bytes(t)), db = span_of(tokens, experts, ldd, c_elem_bytes(d_type));
    if (xb < 0 || db < 0) return TCM_ERR_INVALID_VALUE;
    const int64_t pairs = tokens * topk * 4;
    const Region out[1] = {{D, db}};
    const Region in[6] = {{logits, xb}, {dweights ? ids : nullptr, pairs}, {dweights, pairs}, {mask, tokens},
                          {dlosses ? counts : nullptr, (experts + 1) * 4}, {dlosses, 8}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    RouteGradArgs a{};
    a.x = logits;
    a.tokens = tokens;
    a.ldx = ldx;
    a.experts = (int)experts;
    a.topk = (int)topk;
    a.sigmoid = (flags & TCM_ROUTE_SIGMOID) != 0;
    a.norm = (flags & TCM_ROUTE_NORM) != 0;
    a.d_type = d_type;
    a.scale = scale;
    a.ids = ids;
    a.mask = mask;
    a.dweights = topk > 0 ? dweights : nullptr;
    a.counts = counts;
    a.dlosses = dlosses;
    a.d = D;
    a.ldd = ldd;
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=route_grad tokens=%lld experts=%lld topk=%lld dtype=%d%s%s%s", (long long)v[0], (long long)v[1],
                     (long long)v[2], (int)v[3], v[4] ? " sigmoid=1" : "", v[5] ? " norm=1" : "", v[6] ? " mask=1" : "");
        },
        {tokens, experts, topk, t, a.sigmoid, a.norm, mask != nullptr});
    return done(launch_route_grad(t, a, stream));
}

}  // namespace
}  // namespace tcm

using namespace tcm;

extern "C" {

int tcm_moe_balance(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, const int32_t* ids,
                    const uint8_t* mask, int32_t* counts, float* losses, void* stream) {
    return guarded([&] { return balance_impl(tokens, experts, topk, logits, ldx, dtype, ids, mask, counts, losses, stream); });
}

int tcm_moe_route_grad(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, float scale,
                       const int32_t* ids, const uint8_t* mask, const float* dweights, const int32_t* counts, const float* dlosses,
                       void* D, int64_t ldd, void* stream) {
    return guarded([&] {
        return route_grad_impl(tokens, experts, topk, logits, ldx, dtype, scale, ids, mask, dweights, counts, dlosses, D, ldd, stream);
    });
}

}  // extern "C"
