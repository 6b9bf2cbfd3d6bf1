"""Refusals and empty calls of the 8-bit product, its quantiser, the router and the expert layer (no GPU needed: every
check runs before any HIP call)."""
import pytest

import tensor_core_mixed_amd as T

INV, OK, NOSUP = T.TCM_ERR_INVALID_VALUE, T.TCM_OK, T.TCM_ERR_NOT_SUPPORTED
X, Q, S, QT, ST, Y, Z, W = (0x10000000 * i for i in range(1, 9))  # far apart, never read


def quant(**kw):
    a = dict(rows=100, cols=200, X=X, ldx=200, dtype=T.TCM_BF16_F32, Q=Q, ldq=208, S=S, lds=100, QT=QT, ldqt=112, ST=ST, ldst=200)
    a.update(kw)
    return T.tcm_quantize_fp8(a["rows"], a["cols"], a["X"], a["ldx"], a["dtype"], a["Q"], a["ldq"], a["S"], a["lds"], a["QT"],
                              a["ldqt"], a["ST"], a["ldst"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(ldx=199), dict(ldq=199), dict(lds=99), dict(ldqt=99), dict(ldst=199),
    dict(dtype=T.TCM_I8_I32), dict(dtype=T.TCM_E4M3_F32), dict(dtype=T.TCM_BF16_F32 | T.TCM_C_F16), dict(X=None), dict(S=None),
    dict(ST=None), dict(Q=None, QT=None), dict(S=S + 2), dict(ST=ST + 1), dict(Q=X + 8), dict(QT=Q + 100), dict(S=Q), dict(ST=S),
    dict(S=X + 40), dict(dtype=T.TCM_F32_F32 | T.TCM_BLOCK_TILE, lds=1), dict(dtype=T.TCM_F32_F32 | T.TCM_BLOCK_TILE, ldst=0),
    dict(ldx=1 << 62),
])
def test_quantize_refuses(kw):
    assert quant(**kw) == INV


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0, X=None, Q=None, QT=None)])
def test_quantize_empty(kw):
    assert quant(**kw) == OK


def gemm(**kw):
    a = dict(M=64, N=300, K=500, A=X, lda=512, SA=S, ldsa=64, B=Y, ldb=512, SB=ST, ldsb=4, C=Z, ldc=300, dtype=T.TCM_E4M3_F32,
             bias=W, epi=T.TCM_EPI_BIAS)
    a.update(kw)
    return T.tcm_gemm_fp8(a["M"], a["N"], a["K"], a["A"], a["lda"], a["SA"], a["ldsa"], a["B"], a["ldb"], a["SB"], a["ldsb"],
                          a["C"], a["ldc"], a["dtype"], a["bias"], a["epi"], None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(lda=499), dict(ldb=499), dict(ldc=299), dict(ldsa=63), dict(ldsb=3),
    dict(dtype=T.TCM_F16_F32), dict(dtype=T.TCM_E4M3_F32 | T.TCM_A_COLMAJOR), dict(dtype=T.TCM_E4M3_F32 | T.TCM_C_F16 | T.TCM_C_BF16),
    dict(dtype=T.TCM_E4M3_F32 | T.TCM_B_ROW_SCALES, ldsb=299), dict(dtype=T.TCM_E4M3_F32 | T.TCM_Q_E5M2), dict(A=None), dict(B=None),
    dict(SA=None), dict(SB=None), dict(C=None), dict(bias=None), dict(epi=8), dict(epi=-1), dict(SA=S + 2), dict(SB=ST + 3),
    dict(bias=W + 1), dict(C=X), dict(C=Y + 64), dict(C=S), dict(C=ST), dict(C=W), dict(lda=1 << 61),
])
def test_gemm_refuses(kw):
    assert gemm(**kw) == INV


@pytest.mark.parametrize("kw", [dict(M=0, C=None, A=None), dict(N=0, C=None, B=None)])
def test_gemm_empty(kw):
    assert gemm(**kw) == OK


def test_gemm_types_stay_out_of_the_other_entry_points():
    assert T.tcm_gemm(8, 8, 8, X, 8, Y, 8, Z, 8, T.TCM_E4M3_F32, None, 0, None) == INV


def route(**kw):
    a = dict(tokens=10, experts=64, topk=6, x=X, ldx=64, dtype=T.TCM_F32_F32, bias=Y, scale=1.0, ids=Q, weights=S)
    a.update(kw)
    return T.tcm_moe_route(a["tokens"], a["experts"], a["topk"], a["x"], a["ldx"], a["dtype"], a["bias"], a["scale"], a["ids"],
                           a["weights"], None)


@pytest.mark.parametrize("kw,st", [
    (dict(tokens=-1), INV), (dict(experts=-1), INV), (dict(topk=-1), INV), (dict(topk=65), INV), (dict(ldx=63), INV),
    (dict(dtype=T.TCM_I8_I32), INV), (dict(dtype=T.TCM_F32_F32 | T.TCM_BLOCK_TILE), INV), (dict(x=None), INV), (dict(ids=None), INV),
    (dict(weights=None), INV), (dict(ids=Q + 2), INV), (dict(bias=Y + 1), INV), (dict(weights=S + 1), INV), (dict(ids=X), INV),
    (dict(weights=Q + 16), INV), (dict(weights=Y), INV), (dict(experts=1025, ldx=1025), NOSUP),
    (dict(experts=80, ldx=80, topk=65), NOSUP), (dict(tokens=0, x=None), OK), (dict(topk=0, ids=None), OK),
])
def test_route_refuses(kw, st):
    assert route(**kw) == st


def moe(**kw):
    a = dict(tokens=4, hidden=256, inter=128, experts=8, topk=2, x=X, ldx=256, ids=Q, weights=S, w1=Y, s1=ST, w2=QT, s2=W, out=Z,
             ldo=256, dtype=T.TCM_BF16_F32 | T.TCM_C_BF16 | T.TCM_W_E4M3)
    a.update(kw)
    return T.tcm_moe(a["tokens"], a["hidden"], a["inter"], a["experts"], a["topk"], a["x"], a["ldx"], a["ids"], a["weights"],
                     a["w1"], a["s1"], a["w2"], a["s2"], a["out"], a["ldo"], a["dtype"], None)


@pytest.mark.parametrize("kw,st", [
    (dict(tokens=-1), INV), (dict(hidden=-1), INV), (dict(inter=-1), INV), (dict(experts=-1), INV), (dict(topk=-1), INV),
    (dict(tokens=1 << 31), INV), (dict(ldx=255), INV), (dict(ldo=255), INV), (dict(dtype=T.TCM_F32_F32), INV),
    (dict(dtype=T.TCM_BF16_F32), INV), (dict(dtype=T.TCM_F16_F32 | T.TCM_C_BF16), INV),
    (dict(dtype=T.TCM_BF16_F32 | T.TCM_C_BF16 | T.TCM_ROUTE_NORM), INV), (dict(x=None), INV), (dict(ids=None), INV),
    (dict(weights=None), INV), (dict(w1=None), INV), (dict(w2=None), INV), (dict(s1=None), INV), (dict(s2=None), INV),
    (dict(out=None), INV), (dict(ids=Q + 1), INV), (dict(weights=S + 2), INV), (dict(s1=ST + 2), INV), (dict(out=X + 64), INV),
    (dict(out=Y), INV), (dict(out=QT), INV), (dict(out=Q), INV), (dict(out=S), INV), (dict(out=ST), INV), (dict(out=W), INV),
    (dict(tokens=0, x=None), OK), (dict(hidden=0, out=None), OK),
])
def test_moe_refuses(kw, st):
    assert moe(**kw) == st


@pytest.mark.parametrize("key,default,allowed,refused", [
    ("fp8_config", -1, (-1, 0, 3, 4, 5), (-2, 6, 1 << 32)), ("fp8_split", 0, (0, 1, 64), (-1, 65, 1 << 32))])
def test_options(key, default, allowed, refused):
    assert T.tcm_get_option(key) == default
    try:
        for value in allowed:
            assert T.tcm_set_option(key, value) == OK and T.tcm_get_option(key) == value
        for value in refused:
            assert T.tcm_set_option(key, value) == INV and T.tcm_get_option(key) == allowed[-1]
    finally:
        assert T.tcm_set_option(key, default) == OK
