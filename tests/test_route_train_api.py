"""Refusals and empty calls of the router's losses and gradient (no GPU needed: every check runs before any HIP call)."""
import pytest

import tensor_core_mixed_amd as T

INV, OK, NOSUP = T.TCM_ERR_INVALID_VALUE, T.TCM_OK, T.TCM_ERR_NOT_SUPPORTED
X, I, M, N, F, D, G = (0x10000000 * i for i in range(1, 8))  # far apart, never read


def balance(**kw):
    a = dict(tokens=10, experts=64, topk=6, x=X, ldx=64, dtype=T.TCM_F32_F32, ids=I, mask=M, counts=N, losses=F)
    a.update(kw)
    return T.tcm_moe_balance(a["tokens"], a["experts"], a["topk"], a["x"], a["ldx"], a["dtype"], a["ids"], a["mask"], a["counts"],
                             a["losses"], None)


@pytest.mark.parametrize("kw,st", [
    (dict(tokens=-1), INV), (dict(experts=-1), INV), (dict(topk=-1), INV), (dict(topk=65), INV), (dict(ldx=63), INV),
    (dict(tokens=1 << 31), INV), (dict(dtype=T.TCM_I8_I32), INV), (dict(dtype=T.TCM_F32_F32 | T.TCM_ROUTE_NORM), INV),
    (dict(dtype=T.TCM_F32_F32 | T.TCM_C_BF16), INV), (dict(x=None), INV), (dict(ids=None), INV), (dict(counts=None), INV),
    (dict(losses=None), INV), (dict(ids=I + 2), INV), (dict(counts=N + 1), INV), (dict(losses=F + 2), INV), (dict(counts=X), INV),
    (dict(losses=X + 8), INV), (dict(counts=I), INV), (dict(losses=N + 64 * 4), INV), (dict(counts=M), INV), (dict(ldx=1 << 60), INV),
    (dict(experts=1025, ldx=1025), NOSUP), (dict(experts=80, ldx=80, topk=65), NOSUP), (dict(tokens=1 << 30, topk=2), NOSUP),
])
def test_balance_refuses(kw, st):
    assert balance(**kw) == st


def grad(**kw):
    a = dict(tokens=10, experts=64, topk=6, x=X, ldx=64, dtype=T.TCM_F32_F32, scale=1.0, ids=I, mask=M, dweights=G, counts=N,
             dlosses=F, D=D, ldd=64)
    a.update(kw)
    return T.tcm_moe_route_grad(a["tokens"], a["experts"], a["topk"], a["x"], a["ldx"], a["dtype"], a["scale"], a["ids"], a["mask"],
                                a["dweights"], a["counts"], a["dlosses"], a["D"], a["ldd"], None)


@pytest.mark.parametrize("kw,st", [
    (dict(tokens=-1), INV), (dict(experts=-1), INV), (dict(topk=-1), INV), (dict(topk=65), INV), (dict(ldx=63), INV), (dict(ldd=63), INV),
    (dict(tokens=1 << 31), INV), (dict(dtype=T.TCM_I8_I32), INV), (dict(dtype=T.TCM_F32_F32 | T.TCM_BLOCK_TILE), INV),
    (dict(dtype=T.TCM_F32_F32 | T.TCM_C_BF16 | T.TCM_C_F16), INV), (dict(x=None), INV), (dict(ids=None), INV), (dict(D=None), INV),
    (dict(counts=None), INV), (dict(ids=I + 2), INV), (dict(dweights=G + 1), INV), (dict(counts=N + 1), INV), (dict(dlosses=F + 2), INV),
    (dict(D=X), INV), (dict(D=I), INV), (dict(D=G), INV), (dict(D=N), INV), (dict(D=F), INV), (dict(D=M), INV), (dict(ldd=1 << 60), INV),
    (dict(experts=1025, ldx=1025, ldd=1025), NOSUP), (dict(experts=80, ldx=80, ldd=80, topk=65), NOSUP), (dict(tokens=0, x=None), OK),
    (dict(experts=0, topk=0, D=None), OK),
])
def test_grad_refuses(kw, st):
    assert grad(**kw) == st
