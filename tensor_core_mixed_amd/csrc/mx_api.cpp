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
    // (a launch counts its threads in 32 bits)
    if (((M + 63) / 64) * ((N + 63) / 64) >= ((int64_t)1 << 24)) return TCM_ERR_NOT_SUPPORTED;
    set_last_plan(
        [](char* buf, size_t n, const int64_t* v) {
            snprintf(buf, n, "kernel=fp4_generic M=%lld N=%lld K=%lld", (long long)v[0], (long long)v[1], (long long)v[2]);
        },
        {M, N, K});
    return done(launch_fp4_generic(a, stream));
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
