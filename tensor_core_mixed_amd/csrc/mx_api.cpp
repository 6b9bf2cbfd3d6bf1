// C ABI of the block-scaled 4-bit product and its quantiser (declared in
// include/tcm.h): argument checks and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "api_util.h"
#include "lowp.h"
#include "tcm_internal.h"

namespace tcm {
namespace {

// rows x cols 4-bit values in rows of ld bytes, and their scale words in rows of lds; false past 2^62 bytes
bool mx_spans(int64_t rows, int64_t cols, int64_t ld, int64_t lds, int64_t* q, int64_t* s) {
    *q = span_of(rows, mx_bytes(cols), ld, 1);
    *s = span_of(mx_words(cols), rows, lds, 4);
    return *q >= 0 && *s >= 0;
}

int mx_quantize_impl(int64_t rows, int64_t cols, const void* x, int64_t ldx, int dtype, void* q, int64_t ldq, uint32_t* s,
                     int64_t lds, void* qt, int64_t ldqt, uint32_t* st, int64_t ldst, void* stream) {
    if (dtype != TCM_F16_F32 && dtype != TCM_BF16_F32 && dtype != TCM_F32_F32) return TCM_ERR_INVALID_VALUE;
    if (rows < 0 || cols < 0 || rows >= kDim || cols >= kDim || ldx < std::max<int64_t>(cols, 1)) return TCM_ERR_INVALID_VALUE;
    if (q && (ldq < std::max<int64_t>(mx_bytes(cols), 1) || lds < std::max<int64_t>(rows, 1))) return TCM_ERR_INVALID_VALUE;
    if (qt && (ldqt < std::max<int64_t>(mx_bytes(rows), 1) || ldst < std::max<int64_t>(cols, 1))) return TCM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!x || (!q && !qt) || (q && !s) || (qt && !st)) return TCM_ERR_INVALID_VALUE;
    if ((q && !word_aligned(s)) || (qt && !word_aligned(st))) return TCM_ERR_INVALID_VALUE;
    const int64_t xb = span_of(rows, cols, ldx, elem_bytes(dtype));
    int64_t qb = 0, sb = 0, qtb = 0, stb = 0;
    if (xb < 0 || (q && !mx_spans(rows, cols, ldq, lds, &qb, &sb)) || (qt && !mx_spans(cols, rows, ldqt, ldst, &qtb, &stb)))
        return TCM_ERR_INVALID_VALUE;
    const Region out[4] = {{q, qb}, {qt, qtb}, {q ? s : nullptr, sb}, {qt ? st : nullptr, stb}}, in[1] = {{x, xb}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    MxQuantArgs a{};
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
            snprintf(buf, n, "kernel=mx_quantize rows=%lld cols=%lld dtype=%d out=%s", (long long)v[0], (long long)v[1], (int)v[2],
                     v[3] ? (v[4] ? "both" : "rows") : "cols");
        },
        {rows, cols, dtype, q != nullptr, qt != nullptr});
    return done(launch_mx_quantize(dtype, a, stream));
}

int mx_dequantize_impl(int64_t rows, int64_t cols, const void* q, int64_t ldq, const uint32_t* s, int64_t lds, void* x, int64_t ldx,
                       int dtype, void* stream) {
    if (dtype != TCM_F16_F32 && dtype != TCM_BF16_F32 && dtype != TCM_F32_F32) return TCM_ERR_INVALID_VALUE;
    if (rows < 0 || cols < 0 || rows >= kDim || cols >= kDim || ldx < std::max<int64_t>(cols, 1)) return TCM_ERR_INVALID_VALUE;
    if (ldq < std::max<int64_t>(mx_bytes(cols), 1) || lds < std::max<int64_t>(rows, 1)) return TCM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    if (!x || !q || !s || !word_aligned(s)) return TCM_ERR_INVALID_VALUE;
    const int64_t xb = span_of(rows, cols, ldx, elem_bytes(dtype));
    int64_t qb = 0, sb = 0;
    if (xb < 0 || !mx_spans(rows, cols, ldq, lds, &qb, &sb)) return TCM_ERR_INVALID_VALUE;
    const Region out[1] = {{x, xb}}, in[2] = {{q, qb}, {s, sb}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    MxQuantArgs a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.q = (unsigned char*)const_cast<void*>(q);
    a.ldq = ldq;
    a.s = const_cast<uint32_t*>(s);
    a.lds = lds;
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=mx_dequantize rows=%lld cols=%lld dtype=%d", (long long)v[0], (long long)v[1], (int)v[2]);
        },
        {rows, cols, dtype});
    return done(launch_mx_dequantize(dtype, a, stream));
}

// Sizes, strides and alignment that the fast kernels take: 16-byte rows of A
// and B, and a macro tile's rows within a buffer descriptor's range (2^30).
bool fp4_tiles_fit(const Fp4Args& a) {
    const int64_t lim = ((int64_t)1 << 30) / 256;
    return a.K > 0 && !((uintptr_t)a.A & 15) && !((uintptr_t)a.B & 15) && !(a.lda & 15) && !(a.ldb & 15) && a.lda < lim && a.ldb < lim;
}
// The macro tile and the k ranges of a product by a model of its time, in
// microseconds: the launch; for every round of workgroups a fill of its
// pipelines and its K-steps, whose time grows from `lone` to `shared` as the
// chip fills, or the operands' way from memory where that is longer; C's or
// the partial tiles' way out; and for a split the sum's launch, each share's
// part of it and the partial tiles' way back.  Fitted to products of 1 to 8192
// rows.
struct Fp4Plan {
    int config, split;
};
Fp4Plan plan_fp4(const Fp4Args& a, const LowpOpts& o) {
    static constexpr struct {
        int per_cu;
        double lone, shared;
    } kStep[kNumFp4Tiles] = {{1, 1.28, 1.68}, {1, 0.7, 1.03}, {2, 0.6, 1.2}, {2, 0.31, 0.72}};
    // a launch counts its threads in 32 bits: so many workgroups of a product, at most 512 threads each, and of a sum, 256
    // threads for 1024 outputs
    constexpr int64_t kMaxWgs = (int64_t)1 << 22, kMaxSums = ((int64_t)1 << 24) - 1;
    constexpr double kFixed = 3.0, kRound = 3.0, kSum = 2.5, kShare = 0.25, kBytesPerUs = 5e6;
    Fp4Plan best{kFp4Generic, 1};
    if (!fp4_tiles_fit(a) || o.fp4_config == kFp4Generic) return best;
    const int64_t steps = (a.K + 255) / 256;
    const double memory = (double)(a.M + a.N) * (double)a.K * 0.53 / kBytesPerUs;
    double best_t = 1e30;
    const int forced = o.fp4_config;
    for (int c = 0; c < kNumFp4Tiles; ++c) {
        if (forced >= 0 && forced < kNumFp4Tiles && c != forced) continue;
        const Fp4Tile& t = kFp4Tiles[c];
        const int64_t tiles = ((a.M + t.bm - 1) / t.bm) * ((a.N + t.bn - 1) / t.bn);
        const int64_t slots = 256 * kStep[c].per_cu;
        const bool sums = tiles * (t.bm * t.bn / 1024) <= kMaxSums;
        const int64_t most = std::min({sums ? (int64_t)kFp4MaxSplit : 1, steps, (kMaxWgs - 1) / tiles});
        for (int s = 1; s <= most; ++s) {
            if (o.fp4_split && s != std::min<int64_t>(o.fp4_split, most)) continue;
            const int64_t wgs = tiles * s, rest = wgs % slots;
            const double step = (double)(wgs / slots) * kStep[c].shared +
                                (rest == 0 ? 0 : kStep[c].lone + (kStep[c].shared - kStep[c].lone) * (double)rest / (double)slots);
            const double rounds = (double)((wgs + slots - 1) / slots);
            const double out = (double)wgs * t.bm * t.bn * (s > 1 ? 4 : c_elem_bytes(a.c_type)) / kBytesPerUs;
            const double time = kFixed + std::max(rounds * kRound + (double)((steps + s - 1) / s) * step, memory) + out +
                                (s > 1 ? kSum + kShare * s + 4.0 * s * (double)a.M * (double)a.N / kBytesPerUs : 0);
            if (time < best_t) best_t = time, best = {c, s};
        }
    }
    // Few rows: a workgroup's waves take a step each at a time, rows cost reads of A from the caches.
    if (forced < 0 ? a.M <= kFp4SkinnyRows : forced == kFp4Skinny) {
        static constexpr double kBlock[4] = {1.0, 1.3, 1.9, 2.0}, kFixedFew = 4.5, kSumFew = 4;
        const int64_t blocks_m = (a.M + kFp4SkinnyRows - 1) / kFp4SkinnyRows;
        const int64_t wgs = blocks_m * ((a.N + kFp4SkinnyCols - 1) / kFp4SkinnyCols);
        const double round = kBlock[std::min<int64_t>((a.M + blocks_m * 16 - 1) / (blocks_m * 16), 4) - 1];
        // (1024 outputs a workgroup: the sum's launch holds what this one does)
        const int64_t most = std::min({(int64_t)kFp4MaxSplit, steps, (kMaxWgs - 1) / wgs});
        for (int s = 1; s <= most; ++s) {
            if (o.fp4_split && s != std::min<int64_t>(o.fp4_split, most)) continue;
            const double time = kFixedFew + std::max((double)((wgs * s + 255) / 256) * (double)((steps + 8 * s - 1) / (8 * s)) * round, memory) +
                                (s > 1 ? kSumFew + kShare * s + 8.0 * s * (double)a.M * (double)a.N / kBytesPerUs : 0);
            if (time < best_t || forced == kFp4Skinny && best.config != kFp4Skinny) best_t = time, best = {kFp4Skinny, s};
        }
    }
    return best;
}

int gemm_mx_impl(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const uint32_t* sa, int64_t ldsa, const void* B,
                 int64_t ldb, const uint32_t* sb, int64_t ldsb, void* C, int64_t ldc, int dtype, const float* bias, int epilogue,
                 void* stream) {
    const int flags = dtype & ~0xff;
    if ((dtype & 0xff) != TCM_MXFP4_F32 || (flags & ~(TCM_C_F16 | TCM_C_BF16))) return TCM_ERR_INVALID_VALUE;
    if ((flags & TCM_C_F16) && (flags & TCM_C_BF16)) return TCM_ERR_INVALID_VALUE;
    if (epilogue < 0 || epilogue > (TCM_EPI_BIAS | TCM_EPI_RELU | TCM_EPI_ACCUM)) return TCM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || M >= kDim || N >= kDim || K >= kDim) return TCM_ERR_INVALID_VALUE;
    const int64_t row = std::max<int64_t>(mx_bytes(K), 1);
    if (lda < row || ldb < row || ldc < std::max<int64_t>(N, 1)) return TCM_ERR_INVALID_VALUE;
    if (ldsa < std::max<int64_t>(M, 1) || ldsb < std::max<int64_t>(N, 1)) return TCM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) {
        set_last_plan("empty problem");
        return TCM_OK;
    }
    const bool use_bias = epilogue & TCM_EPI_BIAS;
    if (!C || (use_bias && !bias) || (K > 0 && (!A || !B || !sa || !sb))) return TCM_ERR_INVALID_VALUE;
    if (!word_aligned(sa) || !word_aligned(sb) || (use_bias && !word_aligned(bias))) return TCM_ERR_INVALID_VALUE;
    const int c_type = (flags & TCM_C_F16) ? C_F16 : ((flags & TCM_C_BF16) ? C_BF16 : C_ACC);
    const int64_t cb = span_of(M, N, ldc, c_elem_bytes(c_type));
    int64_t ab = 0, bb = 0, sab = 0, sbb = 0;
    if (cb < 0 || !mx_spans(M, K, lda, ldsa, &ab, &sab) || !mx_spans(N, K, ldb, ldsb, &bb, &sbb)) return TCM_ERR_INVALID_VALUE;
    const Region out[1] = {{C, cb}}, in[5] = {{A, ab}, {B, bb}, {sa, sab}, {sb, sbb}, {use_bias ? bias : nullptr, N * 4}};
    if (!disjoint(out, in)) return TCM_ERR_INVALID_VALUE;
    Fp4Args a{};
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
    a.has_bias = use_bias;
    a.relu = (epilogue & TCM_EPI_RELU) != 0;
    a.accum = (epilogue & TCM_EPI_ACCUM) != 0;
    a.c_type = c_type;
    a.c_vec = ((uintptr_t)C & 15) == 0 && ((ldc * c_elem_bytes(c_type)) & 15) == 0;
    const Fp4Plan pl = plan_fp4(a, lowp_opts());
    if (pl.config == kFp4Generic) {
        // (a launch counts its threads in 32 bits)
        if (((M + 63) / 64) * ((N + 63) / 64) >= ((int64_t)1 << 24)) return TCM_ERR_NOT_SUPPORTED;
        set_last_plan(
            [](char* buf, size_t n, const int64_t* v) {
                snprintf(buf, n, "kernel=fp4_generic M=%lld N=%lld K=%lld", (long long)v[0], (long long)v[1], (long long)v[2]);
            },
            {M, N, K});
        return done(launch_fp4_generic(a, stream));
    }
    const bool skinny = pl.config == kFp4Skinny;
    const int64_t blocks_m = (M + kFp4SkinnyRows - 1) / kFp4SkinnyRows;
    const Fp4Tile t = skinny ? Fp4Tile{(int)((M + blocks_m * 16 - 1) / (blocks_m * 16)) * 16, kFp4SkinnyCols, 1, 1, 0} : kFp4Tiles[pl.config];
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
            snprintf(buf, n, "kernel=fp4_%s tile=%dx%d tiles=%lld split=%d M=%lld N=%lld K=%lld", v[0] ? "skinny" : "tile", (int)v[1],
                     (int)v[2], (long long)v[3], (int)v[4], (long long)v[5], (long long)v[6], (long long)v[7]);
        },
        {skinny, t.bm, t.bn, tm * tn, a.split, M, N, K});
    return done(skinny ? launch_fp4_skinny(t.bm, a, stream) : launch_fp4_tile(pl.config, a, stream));
}

}  // namespace
}  // namespace tcm

using namespace tcm;

extern "C" {

int tcm_quantize_mxfp4(int64_t rows, int64_t cols, const void* X, int64_t ldx, int dtype, void* Q, int64_t ldq, uint32_t* S,
                       int64_t lds, void* QT, int64_t ldqt, uint32_t* ST, int64_t ldst, void* stream) {
    return guarded([&] { return mx_quantize_impl(rows, cols, X, ldx, dtype, Q, ldq, S, lds, QT, ldqt, ST, ldst, stream); });
}

int tcm_dequantize_mxfp4(int64_t rows, int64_t cols, const void* Q, int64_t ldq, const uint32_t* S, int64_t lds, void* X, int64_t ldx,
                         int dtype, void* stream) {
    return guarded([&] { return mx_dequantize_impl(rows, cols, Q, ldq, S, lds, X, ldx, dtype, stream); });
}

int tcm_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const uint32_t* SA, int64_t ldsa, const void* B,
                   int64_t ldb, const uint32_t* SB, int64_t ldsb, void* C, int64_t ldc, int dtype, const float* bias, int epilogue,
                   void* stream) {
    return guarded([&] { return gemm_mx_impl(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, dtype, bias, epilogue, stream); });
}

}  // extern "C"
