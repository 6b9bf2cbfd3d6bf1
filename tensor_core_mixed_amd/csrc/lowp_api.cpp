// C ABI of the block-scaled 8-bit product, its quantiser, the expert router
// and the mixture-of-experts layer (declared in include/tcm.h): argument
// checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "../../include/tcm.h"
#include "api_util.h"
#include "lowp.h"
#include "tcm_internal.h"

namespace tcm {
namespace {

int quantize_impl(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, void* q, int64_t ldq, float* s,
                  int64_t lds, void* qt, int64_t ldqt, float* st, int64_t ldst, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    if (t != F16 && t != BF16 && t != F32) return TCM_ERR_INVALID_VALUE;
    if (flags & ~(TCM_Q_E5M2 | TCM_BLOCK_TILE)) return TCM_ERR_INVALID_VALUE;
    const bool tile = flags & TCM_BLOCK_TILE;
    if (rows < 0 || cols < 0 || rows >= kDim || cols >= kDim || ldx < std::max<int64_t>(cols, 1)) return TCM_ERR_INVALID_VALUE;
    const int64_t rb = scale_blocks(rows), cb = scale_blocks(cols);
    if (q && (ldq < std::max<int64_t>(cols, 1) || lds < std::max<int64_t>(tile ? cb : rows, 1))) return TCM_ERR_INVALID_VALUE;
    if (qt && (ldqt < std::max<int64_t>(rows, 1) || ldst < std::max<int64_t>(tile ? rb : cols, 1))) return TCM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!x || (!q && !qt) || (q && !s) || (qt && !st)) return TCM_ERR_INVALID_VALUE;
    if ((q && !word_aligned(s)) || (qt && !word_aligned(st))) return TCM_ERR_INVALID_VALUE;
    const int64_t xb = span_of(rows, cols, ldx, elem_bytes(t));
    const int64_t qb = q ? span_of(rows, cols, ldq, 1) : 0, qtb = qt ? span_of(cols, rows, ldqt, 1) : 0;
    const int64_t sb = q ? (tile ? span_of(rb, cb, lds, 4) : span_of(cb, rows, lds, 4)) : 0;
    const int64_t stb = qt ? (tile ? span_of(cb, rb, ldst, 4) : span_of(rb, cols, ldst, 4)) : 0;
    if (xb < 0 || qb < 0 || qtb < 0 || sb < 0 || stb < 0) return TCM_ERR_INVALID_VALUE;
    const Region out[4] = {{q, qb}, {qt, qtb}, {s, sb}, {st, stb}}, in[1] = {{x, xb}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    QuantArgs a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.q = (unsigned char*)q;
    a.ldq = ldq;
    a.s = s;
    a.lds = lds;
    a.qt = (unsigned char*)qt;
    a.ldqt = ldqt;
    a.st = st;
    a.ldst = ldst;
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=quantize rows=%lld cols=%lld dtype=%d e5m2=%d block=%s out=%s", (long long)v[0], (long long)v[1],
                     (int)v[2], (int)v[3], v[4] ? "tile" : "row", v[5] ? (v[6] ? "both" : "rows") : "cols");
        },
        {rows, cols, t, (flags & TCM_Q_E5M2) != 0, tile, q != nullptr, qt != nullptr});
    return done(launch_quantize(t, flags & TCM_Q_E5M2, tile, a, stream));
}

// Sizes, strides and alignment that the tiled kernels take: 16-byte rows of A
// and B, and a macro tile's rows within a buffer descriptor's range (2^30).
bool fp8_tiles_fit(const Fp8Args& a) {
    const int64_t lim = ((int64_t)1 << 30) / 256;
    return a.K > 0 && a.K <= ((int64_t)1 << 30) && !((uintptr_t)a.A & 15) && !((uintptr_t)a.B & 15) && !(a.lda & 15) &&
           !(a.ldb & 15) && a.lda < lim && a.ldb < lim && a.ldsb < ((int64_t)1 << 26);
}
// The macro tile and the k ranges of a product by a model of its time, in
// microseconds: the launch; for every round of workgroups a fill of its
// pipelines and its K-steps, whose time grows from `lone` to `shared` as the
// chip fills, or the operands' way from memory where that is longer; C's or
// the partial tiles' way out; and for a split the sum's launch, each share's
// part of it and the partial tiles' way back.  Fitted to products of 37 to
// 8192 rows, 8-bit and (binary32 C) 16-bit operands.
struct Fp8Plan {
    int config, split;
};
Fp8Plan plan_fp8(const Fp8Args& a, const LowpOpts& o) {
    static constexpr struct {
        int per_cu;
        double lone, shared, lone_wide, shared_wide;
    } kStep[kNumFp8Tiles] = {{1, 1.28, 1.65, 0, 0}, {1, 0.66, 0.93, 1.6, 1.83}, {2, 0.69, 1.04, 1.2, 2.13}, {2, 0.38, 0.63, 0.75, 1.19}};
    // a launch counts its threads in 32 bits: so many workgroups of a product, at most 512 threads each, and of a sum, 256
    // threads for 1024 outputs
    constexpr int64_t kMaxWgs = (int64_t)1 << 22, kMaxSums = ((int64_t)1 << 24) - 1;
    constexpr double kFixed = 3.0, kRound = 3.0, kSum = 2.5, kShare = 0.25, kBytesPerUs = 5e6;
    Fp8Plan best{kFp8Generic, 1};
    if (!fp8_tiles_fit(a) || o.fp8_config == kFp8Generic) return best;
    const bool wide = a.c_type == C_ACC;
    const int64_t steps = scale_blocks(a.K);
    const double memory = (double)(a.M + a.N) * (double)a.K / kBytesPerUs;
    double best_t = 1e30;
    int forced = o.fp8_config;
    if (forced >= 0 && forced < kNumFp8Tiles && wide && !kFp8Tiles[forced].wide) forced = -1;  // (cannot serve: another tile does)
    for (int c = 0; c < kNumFp8Tiles; ++c) {
        const Fp8Tile& t = kFp8Tiles[c];
        if (wide && !t.wide) continue;
        if (forced >= 0 && c != forced) continue;
        const int64_t tiles = ((a.M + t.bm - 1) / t.bm) * ((a.N + t.bn - 1) / t.bn);
        const double lone = wide ? kStep[c].lone_wide : kStep[c].lone, shared = wide ? kStep[c].shared_wide : kStep[c].shared;
        const int64_t slots = 256 * kStep[c].per_cu;
        const bool sums = tiles * (t.bm * t.bn / 1024) <= kMaxSums;
        const int64_t most = std::min({sums ? (int64_t)kFp8MaxSplit : 1, steps, (kMaxWgs - 1) / tiles});
        for (int s = 1; s <= most; ++s) {
            if (o.fp8_split && s != std::min<int64_t>(o.fp8_split, most)) continue;
            const int64_t wgs = tiles * s, rest = wgs % slots;
            const double step = (double)(wgs / slots) * shared + (rest == 0 ? 0 : lone + (shared - lone) * (double)rest / (double)slots);
            const double rounds = (double)((wgs + slots - 1) / slots);
            const double out = (double)wgs * t.bm * t.bn * (s > 1 ? 4 : c_elem_bytes(a.c_type)) / kBytesPerUs;
            const double time = kFixed + std::max(rounds * kRound + (double)((steps + s - 1) / s) * step, memory) + out +
                                (s > 1 ? kSum + kShare * s + 4.0 * s * (double)a.M * (double)a.N / kBytesPerUs : 0);
            if (time < best_t) best_t = time, best = {c, s};
        }
    }
    // Few rows: a workgroup's waves take a block each at a time, rows cost reads of A from the caches.
    if (o.fp8_config < 0 ? a.M <= kFp8SkinnyRows : o.fp8_config == kFp8Skinny) {
        static constexpr double kBlock[4] = {0.87, 1.4, 1.75, 2.6};
        const int64_t blocks_m = (a.M + kFp8SkinnyRows - 1) / kFp8SkinnyRows;
        const int64_t wgs = blocks_m * ((a.N + kFp8SkinnyCols - 1) / kFp8SkinnyCols);
        const double round = kBlock[std::min<int64_t>((a.M + blocks_m * 16 - 1) / (blocks_m * 16), 4) - 1];
        // (1024 outputs a workgroup: the sum's launch holds what this one does)
        const int64_t most = std::min({(int64_t)kFp8MaxSplit, steps, (kMaxWgs - 1) / wgs});
        for (int s = 1; s <= most; ++s) {
            if (o.fp8_split && s != std::min<int64_t>(o.fp8_split, most)) continue;
            const double time = kFixed + std::max((double)((wgs * s + 255) / 256) * (double)((steps + 8 * s - 1) / (8 * s)) * round, memory) +
                                (s > 1 ? kSum + kShare * s + 8.0 * s * (double)a.M * (double)a.N / kBytesPerUs : 0);
            if (time < best_t) best_t = time, best = {kFp8Skinny, s};
        }
    }
    return best;
}

int gemm_fp8_impl(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* sa, int64_t ldsa, const void* B,
                  int64_t ldb, const float* sb, int64_t ldsb, void* C, int64_t ldc, int dtype, const float* bias, int epilogue,
                  void* stream) {
    const int flags = dtype & ~0xff;
    if ((dtype & 0xff) != TCM_E4M3_F32) return TCM_ERR_INVALID_VALUE;
    if (flags & ~(TCM_A_E5M2 | TCM_B_E5M2 | TCM_B_ROW_SCALES | TCM_C_F16 | TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if ((flags & TCM_C_F16) && (flags & TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if (epilogue < 0 || epilogue > (TCM_EPI_BIAS | TCM_EPI_RELU | TCM_EPI_ACCUM)) return TCM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || M >= kDim || N >= kDim || K >= kDim) return TCM_ERR_INVALID_VALUE;
    const bool b_row = flags & TCM_B_ROW_SCALES;
    const int64_t kb = scale_blocks(K), nb = scale_blocks(N);
    if (lda < std::max<int64_t>(K, 1) || ldb < std::max<int64_t>(K, 1) || ldc < std::max<int64_t>(N, 1)) return TCM_ERR_INVALID_VALUE;
    if (ldsa < std::max<int64_t>(M, 1) || ldsb < std::max<int64_t>(b_row ? N : kb, 1)) return TCM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    if (!C || (use_bias && !bias) || (K > 0 && (!A || !B || !sa || !sb))) return TCM_ERR_INVALID_VALUE;
    if (!word_aligned(sa) || !word_aligned(sb) || (use_bias && !word_aligned(bias))) return TCM_ERR_INVALID_VALUE;
    const int c_type = (flags & TCM_C_F16) ? C_F16 : ((flags & TCM_C_BF16) ? C_BF16 : C_ACC);
    const int64_t ab = K ? span_of(M, K, lda, 1) : 0, bb = K ? span_of(N, K, ldb, 1) : 0;
    const int64_t cb = span_of(M, N, ldc, c_elem_bytes(c_type));
    const int64_t sab = span_of(kb, M, ldsa, 4), sbb = b_row ? span_of(kb, N, ldsb, 4) : span_of(nb, kb, ldsb, 4);
    if (ab < 0 || bb < 0 || cb < 0 || sab < 0 || sbb < 0) return TCM_ERR_INVALID_VALUE;
    const Region out[1] = {{C, cb}}, in[5] = {{A, ab}, {B, bb}, {sa, sab}, {sb, sbb}, {use_bias ? bias : nullptr, N * 4}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    Fp8Args a{};
    a.A = (const unsigned char*)A;
    a.B = (const unsigned char*)B;
    a.C = C;
    a.sa = sa;
    a.sb = sb;
    a.bias = bias;
    a.M = M;
    a.N = N;
    a.K = K;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.ldsa = ldsa;
    a.ldsb = ldsb;
    a.a_e5m2 = (flags & TCM_A_E5M2) != 0;
    a.b_e5m2 = (flags & TCM_B_E5M2) != 0;
    a.b_row = b_row;
    a.has_bias = use_bias;
    a.relu = (epilogue & TCM_EPI_RELU) != 0;
    a.accum = (epilogue & TCM_EPI_ACCUM) != 0;
    a.c_type = c_type;
    a.c_vec = ((uintptr_t)C & 15) == 0 && ((ldc * c_elem_bytes(c_type)) & 15) == 0;
    const Fp8Plan pl = plan_fp8(a, lowp_opts());
    if (pl.config == kFp8Generic) {
        // (a launch counts its threads in 32 bits)
        if (((M + 63) / 64) * ((N + 63) / 64) >= ((int64_t)1 << 24)) return TCM_ERR_NOT_SUPPORTED;
        set_last_plan(
            [](char* buf, size_t n, const int64_t* v) {
                snprintf(buf, n, "kernel=fp8_generic M=%lld N=%lld K=%lld", (long long)v[0], (long long)v[1], (long long)v[2]);
            },
            {M, N, K});
        return done(launch_fp8_generic(a, stream));
    }
    const bool skinny = pl.config == kFp8Skinny;
    const int64_t blocks_m = (M + kFp8SkinnyRows - 1) / kFp8SkinnyRows;
    const Fp8Tile t = skinny ? Fp8Tile{(int)((M + blocks_m * 16 - 1) / (blocks_m * 16)) * 16, kFp8SkinnyCols, 1, 1, 0, true}
                             : kFp8Tiles[pl.config];
    const int64_t tm = (M + t.bm - 1) / t.bm, tn = (N + t.bn - 1) / t.bn;
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.group_m = 4;
    tile_order_shape(a.tiles_m, a.tiles_n, a.group_m, &a.super_m, &a.super_n);
    a.split = pl.split;
    std::unique_lock<std::mutex> order;
    if (a.split > 1) {
        void* ws = nullptr;
        const int st = workspace_for(stream, (skinny ? M * N : tm * tn * t.bm * t.bn) * a.split * 4, &ws, &order);
        if (st != TCM_OK) return st;
        a.ws = (float*)ws;
    }
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=fp8_%s tile=%dx%d tiles=%lld split=%d M=%lld N=%lld K=%lld", v[0] ? "skinny" : "tile", (int)v[1],
                     (int)v[2], (long long)v[3], (int)v[4], (long long)v[5], (long long)v[6], (long long)v[7]);
        },
        {skinny, t.bm, t.bn, tm * tn, a.split, M, N, K});
    if (skinny) return done(launch_fp8_skinny(t.bm, a, stream));
    const auto launch = a.a_e5m2 ? (a.b_e5m2 ? launch_fp8_tile_e5m2_e5m2 : launch_fp8_tile_e5m2_e4m3)
                                 : (a.b_e5m2 ? launch_fp8_tile_e4m3_e5m2 : launch_fp8_tile_e4m3_e4m3);
    if (launch(pl.config, a, stream) != 0) return TCM_ERR_HIP;
    return done(a.split > 1 ? launch_fp8_tile_sum(pl.config, a, stream) : 0);
}

int route_impl(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, const float* bias,
               float scale, int* ids, float* weights, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    if (t != F16 && t != BF16 && t != F32) return TCM_ERR_INVALID_VALUE;
    if (flags & ~(TCM_ROUTE_SIGMOID | TCM_ROUTE_NORM)) return TCM_ERR_INVALID_VALUE;
    if (tokens < 0 || experts < 0 || topk < 0 || tokens >= ((int64_t)1 << 40) || topk > experts) return TCM_ERR_INVALID_VALUE;
    if (ldx < std::max<int64_t>(experts, 1)) return TCM_ERR_INVALID_VALUE;
    if (experts > kRouteMaxExperts || topk > kRouteMaxTopk) return TCM_ERR_NOT_SUPPORTED;
    if (tokens == 0 || topk == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!logits || !ids || !weights) return TCM_ERR_INVALID_VALUE;
    if (!word_aligned(ids) || !word_aligned(weights) || (bias && !word_aligned(bias))) return TCM_ERR_INVALID_VALUE;
    const int64_t xb = span_of(tokens, experts, ldx, elem_bytes(t));
    if (xb < 0) return TCM_ERR_INVALID_VALUE;
    const Region out[2] = {{ids, tokens * topk * 4}, {weights, tokens * topk * 4}}, in[2] = {{logits, xb}, {bias, experts * 4}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    RouteArgs a{};
    a.x = logits;
    a.tokens = tokens;
    a.ldx = ldx;
    a.experts = (int)experts;
    a.topk = (int)topk;
    a.sigmoid = (flags & TCM_ROUTE_SIGMOID) != 0;
    a.norm = (flags & TCM_ROUTE_NORM) != 0;
    a.bias = bias;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=route tokens=%lld experts=%lld topk=%lld dtype=%d%s%s%s", (long long)v[0], (long long)v[1],
                     (long long)v[2], (int)v[3], v[4] ? " sigmoid=1" : "", v[5] ? " norm=1" : "", v[6] ? " bias=1" : "");
        },
        {tokens, experts, topk, t, a.sigmoid, a.norm, bias != nullptr});
    return done(launch_route(t, a, stream));
}

int moe_impl(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t topk, const void* x, int64_t ldx,
             const int* ids, const float* weights, const void* w1, const float* s1, const void* w2, const float* s2, void* out,
             int64_t ldo, int dtype, void* stream) {
    const int t = dtype & 0xff, flags = dtype & ~0xff;
    const bool w8 = flags & TCM_W_E4M3;
    if (t != F16 && t != BF16) return TCM_ERR_INVALID_VALUE;
    // the output has x's type
    if ((flags & ~TCM_W_E4M3) != (t == F16 ? TCM_C_F16 : TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if (tokens < 0 || hidden < 0 || inter < 0 || experts < 0 || topk < 0) return TCM_ERR_INVALID_VALUE;
    if (tokens >= kDim || hidden >= kDim || inter >= kDim || experts >= kDim || topk >= kDim) return TCM_ERR_INVALID_VALUE;
    if (ldx < std::max<int64_t>(hidden, 1) || ldo < std::max<int64_t>(hidden, 1)) return TCM_ERR_INVALID_VALUE;
    if (tokens == 0 || hidden == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    const bool work = inter > 0 && experts > 0 && topk > 0;
    if (!out || (work && (!x || !ids || !weights || !w1 || !w2 || (w8 && (!s1 || !s2))))) return TCM_ERR_INVALID_VALUE;
    if (work && (!word_aligned(ids) || !word_aligned(weights) || (w8 && (!word_aligned(s1) || !word_aligned(s2)))))
        return TCM_ERR_INVALID_VALUE;
    const int64_t ws = w8 ? 1 : 2, pairs = span_of(tokens, topk, topk, 4);
    const int64_t mat = span_of(hidden, inter, inter, 1), w2b = mat < 0 ? -1 : span_of(experts, mat, mat, ws);
    const int64_t w1b = w2b < 0 || w2b > ((int64_t)1 << 60) ? -1 : 2 * w2b;
    const int64_t xb = span_of(tokens, hidden, ldx, 2), ob = span_of(tokens, hidden, ldo, 2);
    if (pairs < 0 || w1b < 0 || xb < 0 || ob < 0) return TCM_ERR_INVALID_VALUE;
    const int64_t sbytes = w8 && work ? experts * scale_blocks(hidden) * scale_blocks(inter) * 4 : 0;
    const Region o[1] = {{out, ob}};
    const Region in[7] = {{x, work ? xb : 0}, {ids, pairs}, {weights, pairs}, {w1, w1b}, {w2, w2b}, {s1, 2 * sbytes}, {s2, sbytes}};
    if (!disjoint(o, in)) return TCM_ERR_INVALID_VALUE;
    MoeArgs a{};
    a.ldx = ldx;
    a.w1 = w1;
    a.s1 = s1;
    a.w2 = w2;
    a.s2 = s2;
    a.ldo = ldo;
    a.hidden = (int)hidden;
    a.inter = (int)inter;
    a.experts = (int)experts;
    a.topk = work ? (int)topk : 0;
    // whole words in every row: the tiled kernels, in calls of kMoePairs pairs at most
    const int64_t per_word = w8 ? 4 : 2;
    const auto words = [](const void* p) { return ((uintptr_t)p & 3) == 0; };
    const bool tiled = work && topk <= kMoePairs && words(x) && words(w1) && words(w2) && ldx % 2 == 0 && hidden % per_word == 0 &&
                       inter % per_word == 0 && experts * std::max(hidden, inter) < ((int64_t)1 << 26);
    // (a launch counts its threads in 32 bits: the tiled sum has one an output, the others take 2^25 waves at most)
    const int64_t per_token = std::max<int64_t>(hidden, work ? topk * inter : 0);
    const int64_t most = tiled ? std::min<int64_t>(kMoePairs / topk, (((int64_t)1 << 32) - 256) / hidden) : ((int64_t)1 << 25) / per_token;
    const int64_t chunk = std::min(most, tokens);
    if (chunk == 0) return TCM_ERR_NOT_SUPPORTED;
    const int64_t h_bytes = (chunk * a.topk * inter * 4 + 15) & ~(int64_t)15, y_bytes = (chunk * a.topk * hidden * 4 + 15) & ~(int64_t)15;
    std::unique_lock<std::mutex> order;
    const int st = workspace_for(stream, std::max<int64_t>(tiled ? h_bytes + y_bytes + chunk * topk * ((inter + 15) / 16) * 4 : h_bytes, 4), &a.ws,
                                 &order);
    if (st != TCM_OK) return st;
    a.y = (float*)((char*)a.ws + h_bytes);
    a.hmax = (unsigned*)((char*)a.ws + h_bytes + y_bytes);
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=moe_%s tokens=%lld hidden=%lld inter=%lld experts=%lld topk=%lld dtype=%d e4m3=%d",
                     v[0] ? "tile" : "generic", (long long)v[1], (long long)v[2], (long long)v[3], (long long)v[4], (long long)v[5],
                     (int)v[6], (int)v[7]);
        },
        {tiled, tokens, hidden, inter, experts, topk, t, w8});
    for (int64_t t0 = 0; t0 < tokens; t0 += chunk) {
        a.tokens = (int)std::min(chunk, tokens - t0);
        a.x = (const char*)x + t0 * ldx * 2;
        a.ids = ids + t0 * a.topk;
        a.weights = weights + t0 * a.topk;
        a.out = (char*)out + t0 * ldo * 2;
        if ((tiled ? launch_moe_tile : launch_moe_generic)(t, w8, a, stream) != 0) return TCM_ERR_HIP;
    }
    return TCM_OK;
}

}  // namespace
}  // namespace tcm

using namespace tcm;

extern "C" {

int tcm_quantize_fp8(int64_t rows, int64_t cols, const void* X, int64_t ldx, int dtype, void* Q, int64_t ldq, float* S,
                     int64_t lds, void* QT, int64_t ldqt, float* ST, int64_t ldst, void* stream) {
    return guarded([&] { return quantize_impl(rows, cols, X, ldx, dtype, Q, ldq, S, lds, QT, ldqt, ST, ldst, stream); });
}

int tcm_gemm_fp8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA, int64_t ldsa, const void* B,
                 int64_t ldb, const float* SB, int64_t ldsb, void* C, int64_t ldc, int dtype, const float* bias, int epilogue,
                 void* stream) {
    return guarded([&] { return gemm_fp8_impl(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, dtype, bias, epilogue, stream); });
}

int tcm_moe_route(int64_t tokens, int64_t experts, int64_t topk, const void* logits, int64_t ldx, int dtype, const float* bias,
                  float scale, int32_t* ids, float* weights, void* stream) {
    return guarded([&] { return route_impl(tokens, experts, topk, logits, ldx, dtype, bias, scale, ids, weights, stream); });
}

int tcm_moe(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int64_t topk, const void* X, int64_t ldx,
            const int32_t* ids, const float* weights, const void* W1, const float* S1, const void* W2, const float* S2, void* out,
            int64_t ldo, int dtype, void* stream) {
    return guarded([&] {
        return moe_impl(tokens, hidden, inter, experts, topk, X, ldx, ids, weights, W1, S1, W2, S2, out, ldo, dtype, stream);
    });
}

}  // extern "C"
