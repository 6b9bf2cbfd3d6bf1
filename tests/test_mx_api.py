"""Refusals and empty calls of the 4-bit product and its quantiser (no GPU needed: every check runs before any HIP call)."""
import pytest

import tensor_core_mixed_amd as T

INV, OK, NOSUP = T.TCM_ERR_INVALID_VALUE, T.TCM_OK, T.TCM_ERR_NOT_SUPPORTED
X, Q, S, QT, ST, Y, Z, W = (0x10000000 * i for i in range(1, 9))  # far apart, never read


def quant(**kw):
    a = dict(rows=101, cols=203, X=X, ldx=203, dtype=T.TCM_BF16_F32, Q=Q, ldq=102, S=S, lds=101, QT=QT, ldqt=51, ST=ST, ldst=203)
    a.update(kw)
    return T.tcm_quantize_mxfp4(a["rows"], a["cols"], a["X"], a["ldx"], a["dtype"], a["Q"], a["ldq"], a["S"], a["lds"], a["QT"],
                                a["ldqt"], a["ST"], a["ldst"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=1 << 31), dict(ldx=202), dict(ldq=101), dict(lds=100), dict(ldqt=50),
    dict(ldst=202), dict(dtype=T.TCM_I8_I32), dict(dtype=T.TCM_MXFP4_F32), dict(dtype=T.TCM_BF16_F32 | T.TCM_C_F16),
    dict(dtype=T.TCM_BF16_F32 | T.TCM_BLOCK_TILE), dict(X=None), dict(S=None), dict(ST=None), dict(Q=None, QT=None), dict(S=S + 2),
    dict(ST=ST + 1), dict(Q=X + 8), dict(QT=Q + 100), dict(S=Q), dict(ST=S), dict(S=X + 40), dict(ldx=1 << 62), dict(lds=1 << 61),
])
def test_quantize_refuses(kw):
    assert quant(**kw) == INV


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0, X=None, Q=None, QT=None)])
def test_quantize_empty(kw):
    assert quant(**kw) == OK


def back(**kw):
    a = dict(rows=101, cols=203, Q=Q, ldq=102, S=S, lds=101, X=X, ldx=203, dtype=T.TCM_F32_F32)
    a.update(kw)
    return T.tcm_dequantize_mxfp4(a["rows"], a["cols"], a["Q"], a["ldq"], a["S"], a["lds"], a["X"], a["ldx"], a["dtype"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(cols=1 << 31), dict(ldx=202), dict(ldq=101), dict(lds=100), dict(dtype=T.TCM_I8_I32),
    dict(dtype=T.TCM_F32_F32 | T.TCM_C_BF16), dict(X=None), dict(Q=None), dict(S=None), dict(S=S + 3), dict(X=Q), dict(X=S + 8),
    dict(ldx=1 << 61),
])
def test_dequantize_refuses(kw):
    assert back(**kw) == INV


@pytest.mark.parametrize("kw", [dict(rows=0, X=None), dict(cols=0, Q=None)])
def test_dequantize_empty(kw):
    assert back(**kw) == OK


def gemm(**kw):
    a = dict(M=64, N=300, K=501, A=X, lda=251, SA=S, ldsa=64, B=Y, ldb=251, SB=ST, ldsb=300, C=Z, ldc=300, dtype=T.TCM_MXFP4_F32,
             bias=W, epi=T.TCM_EPI_BIAS)
    a.update(kw)
    return T.tcm_gemm_mxfp4(a["M"], a["N"], a["K"], a["A"], a["lda"], a["SA"], a["ldsa"], a["B"], a["ldb"], a["SB"], a["ldsb"],
                            a["C"], a["ldc"], a["dtype"], a["bias"], a["epi"], None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(lda=250), dict(ldb=250), dict(ldc=299), dict(ldsa=63), dict(ldsb=299),
    dict(dtype=T.TCM_F16_F32), dict(dtype=T.TCM_E4M3_F32), dict(dtype=T.TCM_MXFP4_F32 | T.TCM_A_COLMAJOR),
    dict(dtype=T.TCM_MXFP4_F32 | T.TCM_C_F16 | T.TCM_C_BF16), dict(dtype=T.TCM_MXFP4_F32 | T.TCM_B_ROW_SCALES), dict(A=None),
    dict(B=None), dict(SA=None), dict(SB=None), dict(C=None), dict(bias=None), dict(epi=8), dict(epi=-1), dict(SA=S + 2),
    dict(SB=ST + 3), dict(bias=W + 1), dict(C=X), dict(C=Y + 64), dict(C=S), dict(C=ST), dict(C=W), dict(lda=1 << 61),
])
def test_gemm_refuses(kw):
    assert gemm(**kw) == INV


@pytest.mark.parametrize("kw", [dict(M=0, C=None, A=None), dict(N=0, C=None, B=None)])
def test_gemm_empty(kw):
    assert gemm(**kw) == OK


def test_gemm_types_stay_out_of_the_other_entry_points():
    assert T.tcm_gemm(8, 8, 8, X, 8, Y, 8, Z, 8, T.TCM_MXFP4_F32, None, 0, None) == INV
    assert T.tcm_gemm_fp8(8, 8, 8, X, 8, S, 8, Y, 8, ST, 1, Z, 8, T.TCM_MXFP4_F32, None, 0, None) == INV


@pytest.mark.parametrize("key,default,allowed,refused", [
    ("fp4_config", -1, (-1, 0, 3, 4, 5), (-2, 6, 1 << 32)), ("fp4_split", 0, (0, 1, 64), (-1, 65, 1 << 32))])
def test_options(key, default, allowed, refused):
    assert T.tcm_get_option(key) == default
    try:
        for value in allowed:
            assert T.tcm_set_option(key, value) == OK and T.tcm_get_option(key) == value
        for value in refused:
            assert T.tcm_set_option(key, value) == INV and T.tcm_get_option(key) == allowed[-1]
    finally:
        assert T.tcm_set_option(key, default) == OK
