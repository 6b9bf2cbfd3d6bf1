"""The bound on a step's singular values, which chooses the exponents of the orthogonalised update: a call is refused just
where a s + b s^3 + c s^5 passes 2^39, so refusals tell the bound, here beside a dense sampling of the polynomial."""
import numpy as np
import pytest

import host_util

# (a c next to nothing beside b^2 among them: one of the two stationary points is then a difference of near numbers)
COEFFICIENTS = [(2.6, -2.6, c) for c in (0.0, 1e-10, 1e-16, -1e-16, 1e-20, -1e-20, 1e-38)] + [
    (3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (0.0, 1.0, -1e-20), (0.0, -1.0, 3.0), (2.0, 0.0, -1.0), (2.0, 1e-20, -1.0), (2.0, -1e-20, -1.0),
    (1e-20, 2.0, -3.0), (-1.0, 4.0, -3.5), (1.0, 0.0, 0.0), (0.3, 2.0, 5.0), (-2.6, 2.6, 1e-18)]


def largest(coef, r=1.001):
    a, b, c = (float(np.float32(v)) for v in coef)
    s = np.linspace(0, r, 1_000_001)
    return float(np.abs(s * (a + s * s * (b + s * s * c))).max())


def test_bound_is_the_largest_value(tmp_path):
    gen = np.random.default_rng(0)
    draws = [tuple(gen.normal(size=3) * np.exp(gen.normal(size=3) * 3)) for _ in range(100)]
    cases = []
    for coef in COEFFICIENTS + draws:
        for near, fits in ((1.003, False), (0.997, True)):
            g = 2.0 ** 39 / 1.001 / largest(coef) * near
            cases.append((tuple(float(np.float32(v * g)) for v in coef), fits))
    out = host_util.run(tmp_path, f"""
        for coef, fits in {cases}:
            st = T.tcm_orthogonalize(1, 20, 30, at(1), 30, 0, at(2), 30, 0, T.TCM_F32_F32, coef + (0.0, 0.0, 0.0), 0.0, 1.0, None)
            if st != (T.TCM_OK if fits else T.TCM_ERR_NOT_SUPPORTED):
                print(coef, fits, st)
    """)
    assert not out, out
