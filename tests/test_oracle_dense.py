"""The float64 oracle of the atom-wise dense operators: its gradients against
central differences of its own forward, and its values where they are known."""
import numpy as np
import pytest

from oracle import dense as D

ACTS = ("none", "relu", "silu", "gelu")


def _slope(f, v, d, h=1e-5):
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


def test_norm_known_values():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    out = D.norm(x, np.array([1.0, 2.0]), eps=0.0 + 1e-300)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(out["y"][0], [3 / r, 8 / r], rtol=1e-14)
    assert np.all(out["y"][1] == 0.0)


def test_activation_known_values():
    z = np.array([-1.0, 0.0, 2.0])
    np.testing.assert_allclose(D.act(z, "silu"), z / (1 + np.exp(-z)), rtol=1e-14)
    np.testing.assert_allclose(D.act(z, "gelu")[2], 2 * 0.9772498680518208, rtol=1e-14)  # 2 Phi(2)
    assert list(D.act(z, "relu")) == [0.0, 0.0, 2.0]


@pytest.mark.parametrize("with_gsum", [False, True])
def test_norm_gradient_against_differences(with_gsum):
    r = np.random.default_rng(1)
    x, res, w, gy, gs = (r.normal(size=s) for s in ((3, 7), (3, 7), 7, (3, 7), (3, 7)))
    f = D.norm(x, w, res, 1e-3)
    b = D.norm_backward(gy, f["sum"], w, f["rstd"], gs if with_gsum else None)
    through = lambda o: (o["y"] * gy).sum() + ((o["sum"] * gs).sum() if with_gsum else 0.0)
    for _ in range(4):
        d, dw = r.normal(size=x.shape), r.normal(size=w.shape)
        for at in (lambda v: D.norm(v, w, res, 1e-3), lambda v: D.norm(x, w, v, 1e-3)):
            base = x if at(x)["sum"] is not None and np.array_equal(at(x)["sum"], x + res) else res
            assert abs(_slope(lambda v: through(at(v)), base, d) - (b["gx"] * d).sum()) < 1e-7
        assert abs(_slope(lambda v: through(D.norm(x, v, res, 1e-3)), w, dw) - (b["gweight"] * dw).sum()) < 1e-7


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_against_differences(act):
    r = np.random.default_rng(2)
    x, w, bias, gy = (r.normal(size=s) for s in ((4, 5), (6, 5), 6, (4, 6)))
    z = D.linear(x, w, bias)["preact"]
    assert np.abs(z).min() > 1e-3  # away from the corner of relu
    b = D.linear_backward(gy, x, w, z, act)
    loss = lambda x, w, bias: (D.linear(x, w, bias, act)["y"] * gy).sum()
    for _ in range(4):
        dx, dw, db = r.normal(size=x.shape), r.normal(size=w.shape), r.normal(size=bias.shape)
        assert abs(_slope(lambda v: loss(v, w, bias), x, dx) - (b["gx"] * dx).sum()) < 1e-7
        assert abs(_slope(lambda v: loss(x, v, bias), w, dw) - (b["gw"] * dw).sum()) < 1e-7
        assert abs(_slope(lambda v: loss(x, w, v), bias, db) - (b["gbias"] * db).sum()) < 1e-7
