"""The float64 oracle of the orthogonalised update, pinned by the singular value decomposition."""
import numpy as np
import pytest

from oracle import dense as D


@pytest.mark.parametrize("shape", [(1, 1), (5, 9), (9, 5), (12, 12), (1, 7)])
def test_singular_values_follow_the_polynomial(shape):
    """Singular vectors stay, each singular value s of g / |g| goes to s (a + b s^2 + c s^4) at every step."""
    g = np.random.default_rng(1).normal(size=shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    steps = [D.QUINTIC, D.QUINTIC, (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)]
    for a, b, c in steps:
        s = s * (a + b * s ** 2 + c * s ** 4)
    np.testing.assert_allclose(D.orthogonalize(g, steps), (u * s) @ v, atol=1e-12)


def test_converges_to_the_nearest_orthonormal_rows():
    g = np.random.default_rng(2).normal(size=(6, 20))
    u, _, v = np.linalg.svd(g, full_matrices=False)
    np.testing.assert_allclose(D.orthogonalize(g, [(1.875, -1.25, 0.375)] * 25), u @ v, atol=1e-12)


def test_zeros_stay_zeros():
    assert np.all(D.orthogonalize(np.zeros((3, 4))) == 0.0)
