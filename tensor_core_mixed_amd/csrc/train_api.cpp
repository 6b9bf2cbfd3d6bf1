// C ABI of the router's losses and gradient and of the orthogonalised update
// (declared in include/tcm.h): argument checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
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
        const int64_t g = a.groups;
        void* ws = nullptr;
        const int st = workspace_for(stream, 8 + 8 * g + 4 * g * experts + 4 * g * (experts + 1), &ws, &order);
        if (st != TCM_OK) return st;
        a.arrived = (unsigned long long*)ws;
        a.z = (double*)ws + 1;
        a.p = (float*)(a.z + g);
        a.n = (int*)(a.p + g * experts);
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

// The largest |f| among [0, r] of f(s) = a s + b s^3 + c s^5 (in t = s^2: at the ends and where a + 3 b t + 5 c t^2 = 0).
// The two roots are q / (5 c) and a / q with q of one sign's sum: nothing cancels where c is next to nothing and one of
// them lies far away.
double largest_step(double a, double b, double c, double r) {
    const auto f = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + t * c))); };
    double most = f(r * r);
    const auto at = [&](double t) {
        if (t > 0 && t < r * r) most = std::max(most, f(t));
    };
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
        const double q = -0.5 * (3 * b + std::copysign(std::sqrt(d), b));
        if (c != 0) at(q / (5 * c));
        if (q != 0) at(a / q);
    }
    return most;
}
// and of f(s) = b s + c s^2
double largest_square(double b, double c, double r) {
    const auto f = [&](double s) { return std::fabs(s * (b + s * c)); };
    double most = f(r);
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < r) most = std::max(most, f(-b / (2 * c)));
    return most;
}
// The exponent that takes values up to `most` near 2^14, a quarter of binary16's largest.  (What steps_fit lets pass lies
// within these bounds, is zero, or is not finite, as its values are then.)
int exponent_for(double most) {
    if (!(most > 0x1p-80)) return 80;
    if (!(most < 0x1p80)) return -80;
    return 13 - std::ilogb(most);
}
// Whether the bounds on X between the steps (whose square is S's) and on T are such that these exponents hold them.
bool steps_fit(int steps, const float* coef) {
    double most = 1.001;
    const auto in = [](double v, double lo, double hi) { return v == 0 || (v >= lo && v <= hi); };
    for (int k = 0; k < steps; ++k, coef += 3) {
        const double t = largest_square(coef[1], coef[2], most * most);
        most = largest_step(coef[0], coef[1], coef[2], most) * 1.001;
        if (!std::isfinite(t) || !std::isfinite(most)) return true;
        if (!in(t, 0x1p-79, 0x1p79) || (k < steps - 1 && !in(most, 0x1p-39, 0x1p39))) return false;
    }
    return true;
}

// The factors of step k and of the exponents: `most` bounds X's singular values, `ex` is X's exponent.
struct OrthoScale {
    double most = 1.001;  // (the norm bounds them)
    int ex = exponent_for(1.001);
    OrthoStep next(const float* coef, bool end, float scale) {
        const double ca = coef[0], cb = coef[1], cc = coef[2];
        const auto two = [](double v, int e) { return (float)std::ldexp(v, e); };
        const int es = exponent_for(most * most), et = exponent_for(largest_square(cb, cc, most * most) * 1.001);
        most = largest_step(ca, cb, cc, most) * 1.001;
        const int to = end ? 0 : exponent_for(most);
        const double f = end ? (double)scale : 1.0;
        const OrthoStep q{two(1, es - 2 * ex), two(cc, et - 2 * es), two(cb, et - es), two(f, to - et - ex), two(f * ca, to - ex)};
        ex = to;
        return q;
    }
};

// Shorter sides up to 128 (ortho_small.hip)
int ortho_small(OrthoArgs a, int x_type, int64_t batch, int steps, const float* coef, float scale, void* stream) {
    const auto line = [](int64_t x) { return (x + 255) / 256 * 256; };
    const int64_t n = std::min(a.rows, a.cols), m = std::max(a.rows, a.cols), np = ortho_small_rows(n), cw = kOrthoSmallElems / np;
    const int64_t chunks = (m + cw - 1) / cw;
    const bool one = chunks == 1, kept = !one || steps > kOrthoSmallSteps;
    a.slices = one ? 0 : std::min<int64_t>(kOrthoSlices, (a.rows * ((a.cols + 7) / 8) + 1023) / 1024);
    const int64_t state = kept ? chunks * kOrthoSmallElems * 4 : 0, shares = kept ? chunks * np * np * 4 : 0, entry = a.slices * 8 + state + 2 * shares;
    const int64_t part = std::min({batch, std::max<int64_t>(1, kOrthoWorkspace / std::max<int64_t>(entry, 1)), ((int64_t)1 << 22) / chunks});
    void* ws = nullptr;
    std::unique_lock<std::mutex> order;
    if (kept) {
        const int st = workspace_for(stream, part * (state + 2 * shares) + line(part * a.slices * 8), &ws, &order);
        if (st != TCM_OK) return st;
    }
    set_last_plan(
        [](char* buf, size_t len, const int64_t* v) {
            snprintf(buf, len, "kernel=ortho_small batch=%lld rows=%lld cols=%lld dtype=%d steps=%d chunk=%lld chunks=%lld", (long long)v[0],
                     (long long)v[1], (long long)v[2], (int)v[3], (int)v[4], (long long)v[5], (long long)v[6]);
        },
        {batch, a.rows, a.cols, x_type, steps, part, chunks});
    const char *g = (const char*)a.g, *o = (const char*)a.o;
    for (int64_t b = 0; b < batch; b += part) {
        OrthoSmallArgs p{};
        p.g = a;
        p.g.g = g + b * a.stride_g * elem_bytes(x_type);
        p.g.o = (void*)(o + b * a.stride_o * c_elem_bytes(a.o_type));
        p.g.batch = std::min(part, batch - b);
        p.m = m;
        p.n = (int)n;
        p.tall = a.rows > a.cols;
        p.chunks = (int)chunks;
        p.state = (char*)ws;
        float* s[2] = {(float*)((char*)ws + part * state), (float*)((char*)ws + part * (state + shares))};
        p.g.squares = one ? nullptr : (double*)((char*)ws + part * (state + 2 * shares));
        OrthoScale f;
        p.factor = (float)std::ldexp(1.0, f.ex);
        if (!one && launch_ortho_norm(x_type, p.g, stream) != 0) return TCM_ERR_HIP;
        const int each = one ? kOrthoSmallSteps : 1;
        for (int k = 0, turn = 0; k < steps; ++turn) {
            p.first = turn == 0;
            p.steps = p.first && !one ? 0 : std::min(each, steps - k);
            for (int i = 0; i < p.steps; ++i, ++k) p.step[i] = f.next(coef + 3 * k, k == steps - 1, scale);
            p.last = k == steps;
            p.shares_in = s[~turn & 1];
            p.shares_out = s[turn & 1];
            if (launch_ortho_small(x_type, p, stream) != 0) return TCM_ERR_HIP;
        }
    }
    return TCM_OK;
}

int ortho_impl(int64_t batch, int64_t rows, int64_t cols, const void* g, int64_t ldg, int64_t stride_g, void* o, int64_t ldo,
               int64_t stride_o, int dtype, int steps, const float* coef, float eps, float scale, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    if (t != F16 && t != BF16 && t != F32) return TCM_ERR_INVALID_VALUE;
    if ((flags & ~(TCM_C_F16 | TCM_C_BF16)) || ((flags & TCM_C_F16) && (flags & TCM_C_BF16))) return TCM_ERR_INVALID_VALUE;
    if (batch < 0 || rows < 0 || cols < 0 || batch >= kDim || rows >= kDim || cols >= kDim) return TCM_ERR_INVALID_VALUE;
    if (ldg < std::max<int64_t>(cols, 1) || ldo < std::max<int64_t>(cols, 1)) return TCM_ERR_INVALID_VALUE;
    if (stride_g < 0 || stride_o < 0 || stride_g >= ((int64_t)1 << 40) || stride_o >= ((int64_t)1 << 40)) return TCM_ERR_INVALID_VALUE;
    if (steps < 0 || (steps > 0 && !coef) || !(eps >= 0)) return TCM_ERR_INVALID_VALUE;
    if (batch == 0 || rows == 0 || cols == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!g || !o) return TCM_ERR_INVALID_VALUE;
    const int o_type = (flags & TCM_C_F16) ? C_F16 : ((flags & TCM_C_BF16) ? C_BF16 : C_ACC);
    const int64_t ge = span_of(rows, cols, ldg, 1), oe = span_of(rows, cols, ldo, 1);
    if (ge < 0 || oe < 0 || (batch > 1 && stride_o < oe)) return TCM_ERR_INVALID_VALUE;
    const int64_t gb = span_of(batch, ge, stride_g, elem_bytes(t)), ob = span_of(batch, oe, stride_o, c_elem_bytes(o_type));
    if (batch > 1 && stride_g > (((int64_t)1 << 60) - ge) / (batch - 1)) return TCM_ERR_INVALID_VALUE;
    if (gb < 0 || ob < 0) return TCM_ERR_INVALID_VALUE;
    const Region out[1] = {{o, ob}}, in[1] = {{g, gb}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    if (std::max(rows, cols) > kOrthoMaxSize || !steps_fit(steps, coef)) return TCM_ERR_NOT_SUPPORTED;

    const bool tall = rows > cols;
    const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
    OrthoArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.ldg = ldg;
    a.stride_g = stride_g;
    a.ldo = ldo;
    a.stride_o = stride_o;
    a.o_type = o_type;
    a.eps = eps;
    if (steps > 0 && ortho_small_fits(batch, n, m)) {
        a.g = g;
        a.o = o;
        return ortho_small(a, t, batch, steps, coef, scale, stream);
    }
    const auto pad = [](int64_t x) { return (x + 31) / 32 * 32; };
    const auto line = [](int64_t x) { return (x + 255) / 256 * 256; };
    // an entry's parts: X, X transposed twice (read by other tiles while the next is written), S, T
    const int64_t x_bytes = line(n * pad(m) * 4), xt_bytes = line(m * pad(n) * 4), s_bytes = line(n * pad(n) * 4);
    const int64_t entry = steps ? x_bytes + 2 * xt_bytes + 2 * s_bytes : 0;
    // The tile and the k ranges of a product by a model of its time, in microseconds: the launch; for every round of
    // workgroups a fill and the tiles' way out, and its K-steps; for ranges the second launch and the partial tiles' way
    // there and back.  Fitted to products of 768 to 4096 rows.
    struct Plan {
        int cfg, tiles_m, tiles_n, tiles, split;
        int64_t ws;
    };
    const auto plan = [&](int64_t M, int64_t N, int64_t K, int64_t entries, bool sym) {
        static constexpr struct {
            double whole, part, step;
        } kRound[kNumOrthoTiles] = {{12, 8, 1.65}, {10, 6.5, 0.55}, {5, 5, 0.25}};
        constexpr double kLaunch = 3, kSum = 5, kBytesPerUs = 3e6;
        constexpr int64_t kMaxSplit = 32;
        Plan best{};
        double best_t = 1e30;
        for (int c = 0; c < kNumOrthoTiles; ++c) {
            const OrthoTile& x = kOrthoTiles[c];
            const int64_t tm = (M + x.bm - 1) / x.bm, tn = (N + x.bn - 1) / x.bn, tiles = sym ? tm * (tm + 1) / 2 : tm * tn;
            const int64_t all = tiles * entries, ksteps = pad(K) / 32;
            for (int64_t s = 1; s <= std::min(ksteps, kMaxSplit); ++s) {
                const double rounds = (double)((all * s + 255) / 256), bytes = (double)(all * s * x.bm * x.bn * 4);
                const double time = kLaunch + rounds * ((s > 1 ? kRound[c].part : kRound[c].whole) + kRound[c].step * (double)((ksteps + s - 1) / s)) +
                                    (s > 1 ? kSum + bytes / kBytesPerUs : 0);
                if (time < best_t) best_t = time, best = Plan{c, (int)tm, (int)tn, (int)tiles, (int)s, s > 1 ? (int64_t)bytes : 0};
            }
        }
        return best;
    };
    // entries in parts of a call, so that the workspace stays within bounds and a launch within its 32 bits of threads
    const int64_t tiles = std::max(((n + 127) / 128) * ((m + 127) / 128), ((n + 63) / 64) * ((m + 63) / 64));
    const int64_t chunk = std::min({batch, std::max<int64_t>(1, kOrthoWorkspace / std::max<int64_t>(entry, 1)), std::max<int64_t>(1, ((int64_t)1 << 22) / tiles)});
    const Plan ps = plan(n, n, m, chunk, true), pt = plan(n, n, n, chunk, true), px = plan(n, m, n, chunk, false);
    const int64_t slices = std::min<int64_t>(kOrthoSlices, (rows * ((cols + 7) / 8) + 1023) / 1024);
    const int64_t squares = line(chunk * slices * 8), partial = std::max({ps.ws, pt.ws, px.ws});
    void* ws = nullptr;
    std::unique_lock<std::mutex> order;
    const int st = workspace_for(stream, squares + chunk * entry + partial, &ws, &order);
    if (st != TCM_OK) return st;
    set_last_plan(
        [](char* buf, size_t len, const int64_t* v) {
            snprintf(buf, len, "kernel=ortho batch=%lld rows=%lld cols=%lld dtype=%d steps=%d chunk=%lld tile=%d,%d,%d split=%lld", (long long)v[0],
                     (long long)v[1], (long long)v[2], (int)v[3], (int)v[4], (long long)v[5], (int)(v[6] / 100), (int)(v[6] / 10 % 10),
                     (int)(v[6] % 10), (long long)v[7]);
        },
        {batch, rows, cols, t, steps, chunk, 100 * ps.cfg + 10 * pt.cfg + px.cfg, ps.split * 10000 + pt.split * 100 + px.split});
    for (int64_t b = 0; b < batch; b += chunk) {
        const int64_t count = std::min(chunk, batch - b);
        char* base = (char*)ws + squares;
        char *x = base, *xt[2] = {base + x_bytes, base + x_bytes + xt_bytes}, *sq = base + x_bytes + 2 * xt_bytes, *tt = sq + s_bytes;
        a.g = (const char*)g + b * stride_g * elem_bytes(t);
        a.batch = count;
        a.o = (char*)o + b * stride_o * c_elem_bytes(o_type);
        a.rows_pad = pad(rows);
        a.cols_pad = pad(cols);
        a.slices = slices;
        a.squares = (double*)ws;
        a.as_is = tall ? xt[0] : x;
        a.across = tall ? x : xt[0];
        a.entry_bytes = entry;
        OrthoScale f;
        if (launch_ortho_norm(t, a, stream) != 0) return TCM_ERR_HIP;
        if (launch_ortho_start(t, a, steps ? (float)std::ldexp(1.0, f.ex) : scale, steps == 0, stream) != 0) return TCM_ERR_HIP;
        for (int k = 0; k < steps; ++k) {
            const bool end = k == steps - 1;
            const OrthoStep step = f.next(coef + 3 * k, end, scale);
            const auto mul = [&](const Plan& p, int64_t M, int64_t N, int64_t K, bool sym) {
                OrthoMul q{};
                q.entry_bytes = entry;
                q.M = M;
                q.N = N;
                q.k_pad = pad(K);
                q.n_pad = pad(N);
                q.m_pad = pad(M);
                q.batch = (int)count;
                q.symmetric = sym;
                q.tiles = p.tiles;
                q.tiles_m = p.tiles_m;
                q.tiles_n = p.tiles_n;
                q.group_m = 4;
                tile_order_shape(q.tiles_m, q.tiles_n, q.group_m, &q.super_m, &q.super_n);
                q.split = p.split;
                q.ws = (float*)(base + chunk * entry);
                return q;
            };
            OrthoMul q = mul(ps, n, n, m, true);  // S
            q.A = q.B = x;
            q.D = q.E = sq;
            q.alpha = step.s_alpha;
            if (launch_ortho_mul(ps.cfg, q, stream) != 0) return TCM_ERR_HIP;
            q = mul(pt, n, n, n, true);  // T
            q.A = q.B = q.P = sq;
            q.D = q.E = tt;
            q.alpha = step.t_alpha;
            q.beta = step.t_beta;
            if (launch_ortho_mul(pt.cfg, q, stream) != 0) return TCM_ERR_HIP;
            q = mul(px, n, m, n, false);  // X
            q.A = tt;
            q.B = xt[k & 1];
            q.P = x;
            q.D = x;
            q.E = xt[~k & 1];
            q.alpha = step.x_alpha;
            q.beta = step.x_beta;
            if (end) {
                q.out = (char*)a.o;
                q.ld_out = ldo;
                q.stride_out = stride_o;
                q.out_type = o_type;
                q.out_across = tall;
            }
            if (launch_ortho_mul(px.cfg, q, stream) != 0) return TCM_ERR_HIP;
        }
    }
    return TCM_OK;
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

int tcm_orthogonalize(int64_t batch, int64_t rows, int64_t cols, const void* G, int64_t ldg, int64_t stride_g, void* O, int64_t ldo,
                      int64_t stride_o, int dtype, int steps, const float* coefficients, float eps, float scale, void* stream) {
    return guarded([&] {
        return ortho_impl(batch, rows, cols, G, ldg, stride_g, O, ldo, stride_o, dtype, steps, coefficients, eps, scale, stream);
    });
}

}  // extern "C"
