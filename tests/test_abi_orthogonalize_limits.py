"""Coefficients whose largest step lies within [0, 1] (CPU only): the polynomials' turning points are found also where one
of their coefficients is next to nothing beside the others."""
import numpy as np
import pytest

from test_abi_dense import P
from test_abi_orthogonalize import ortho


def largest(a, b, c):
    """What a step takes singular values of [0, 1] to at most, and b s^2 + c s^4, on a fine grid."""
    q = np.linspace(0.0, 1.0, 50001)
    return np.abs(np.sqrt(q) * (a + q * (b + c * q))).max(), np.abs(q * (b + c * q)).max()


STEEP = [(18.5, -15.0, 0.0), (-18.5, 15.0, 0.0), (12.0, -12.0, 0.0), (10.5, -13.5, 0.0)]  # 7.9, 4.6 and 3.56 within, 3.5 at most at 1


@pytest.mark.parametrize("c", [0.0, 1e-300, -1e-300, 1e-20, -1e-20, 1e-16, -1e-16, 1e-14, -1e-14, 1e-10, 1e-6, -1e-6])
@pytest.mark.parametrize("a,b,_", STEEP)
def test_turning_points_are_found(a, b, _, c):
    grown, poly = largest(a, b, c)
    assert grown > 3.52 and poly < 15.01 and abs(a + b + c) <= 3.51
    assert ortho(y=P(1), steps=1, coef=(a, b, c)) == "EEC_ERR_SHAPE"


def test_sets_within_the_limits_pass():
    """Whatever stays within the limits is let through (and then refused for its outputs, which lie over its inputs)."""
    r = np.random.default_rng(0)
    passed = 0
    for _ in range(3000):
        a, b, c = (float(v) for v in r.uniform(-20, 20, 3) * 10.0 ** r.choice([0, -1, -8, -17, -200], 3))
        grown, poly = largest(a, b, c)
        if abs(grown - 3.5) < 1e-3 or abs(poly - 15.0) < 1e-3:
            continue
        ok = grown <= 3.5 and poly <= 15.0
        passed += ok
        assert ortho(y=P(1), steps=1, coef=(a, b, c)) == ("EEC_ERR_ALIAS" if ok else "EEC_ERR_SHAPE"), (a, b, c)
    assert passed > 300
