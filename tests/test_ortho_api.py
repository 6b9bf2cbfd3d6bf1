"""Refusals and empty calls of the orthogonalised update (no GPU needed: every check runs before any HIP call)."""
import pytest

import tensor_core_mixed_amd as T

INV, OK, NOSUP = T.TCM_ERR_INVALID_VALUE, T.TCM_OK, T.TCM_ERR_NOT_SUPPORTED
G, O = 1 << 40, 1 << 50  # far apart, never read
C5 = (3.4445, -4.7750, 2.0315) * 5


def ortho(**kw):
    a = dict(batch=2, rows=30, cols=40, G=G, ldg=41, sg=1300, O=O, ldo=40, so=1200, dtype=T.TCM_BF16_F32, coef=C5, eps=1e-7, scale=1.0)
    a.update(kw)
    return T.tcm_orthogonalize(a["batch"], a["rows"], a["cols"], a["G"], a["ldg"], a["sg"], a["O"], a["ldo"], a["so"], a["dtype"],
                               a["coef"], a["eps"], a["scale"], None)


@pytest.mark.parametrize("kw,st", [
    (dict(batch=-1), INV), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(batch=1 << 31), INV), (dict(rows=1 << 31), INV),
    (dict(ldg=39), INV), (dict(ldo=39), INV), (dict(sg=-1), INV), (dict(so=-1), INV), (dict(so=1199), INV), (dict(sg=1 << 40), INV),
    (dict(so=1 << 40), INV), (dict(dtype=T.TCM_I8_I32), INV), (dict(dtype=T.TCM_F32_F32 | T.TCM_C_F16 | T.TCM_C_BF16), INV),
    (dict(dtype=T.TCM_F32_F32 | T.TCM_ROUTE_NORM), INV), (dict(G=None), INV), (dict(O=None), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(O=G), INV), (dict(O=G + 2 * 1300 + 64), INV), (dict(ldg=1 << 60), INV),
    (dict(rows=1, cols=(1 << 20) - 31, ldg=1 << 20, ldo=1 << 20, so=1 << 20), NOSUP), (dict(batch=0, G=None), OK), (dict(rows=0, O=None), OK),
    (dict(cols=0), OK),
])
def test_refuses(kw, st):
    assert ortho(**kw) == st


def test_coefficients():
    assert T.lib().tcm_orthogonalize(1, 4, 4, G, 4, 16, O, 4, 16, T.TCM_F32_F32, -1, None, 0.0, 1.0, None) == INV
    assert T.lib().tcm_orthogonalize(1, 4, 4, G, 4, 16, O, 4, 16, T.TCM_F32_F32, 2, None, 0.0, 1.0, None) == INV
    with pytest.raises(ValueError):
        ortho(coef=C5[:-1])
