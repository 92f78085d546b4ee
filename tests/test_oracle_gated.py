"""The float64 oracle of the gated layer and of rows in 8 bits: gradients against central differences, values where they are known."""
import numpy as np
import pytest

from oracle import dense as D


@pytest.mark.parametrize("act", ("none", "relu", "silu", "gelu"))
def test_gated_gradient_against_differences(act):
    r = np.random.default_rng(3)
    x, w, bias, gy = (r.normal(size=s) for s in ((4, 5), (12, 5), 12, (4, 6)))
    z = D.gated(x, w, bias, act)["preact"]
    assert np.abs(z[:, :6]).min() > 1e-3  # away from the corner of relu
    b = D.gated_backward(gy, x, w, z, act)
    loss = lambda x, w, bias: (D.gated(x, w, bias, act)["y"] * gy).sum()
    h = 1e-5
    for _ in range(4):
        dx, dw, db = r.normal(size=x.shape), r.normal(size=w.shape), r.normal(size=bias.shape)
        assert abs((loss(x + h * dx, w, bias) - loss(x - h * dx, w, bias)) / (2 * h) - (b["gx"] * dx).sum()) < 1e-7
        assert abs((loss(x, w + h * dw, bias) - loss(x, w - h * dw, bias)) / (2 * h) - (b["gw"] * dw).sum()) < 1e-7
        assert abs((loss(x, w, bias + h * db) - loss(x, w, bias - h * db)) / (2 * h) - (b["gbias"] * db).sum()) < 1e-7


def test_gated_known_values():
    # gate 2, value 3: silu(2) 3, relu(2) 3, and the bilinear 2 x 3; a value of zero stops the gate
    x, w = np.array([[1.0]]), np.array([[2.0], [0.5], [3.0], [0.0]])
    y = lambda act: D.gated(x, w, None, act)["y"][0]
    np.testing.assert_allclose(y("silu"), [6.0 / (1 + np.exp(-2.0)), 0.0], rtol=1e-14)
    np.testing.assert_allclose(y("relu"), [6.0, 0.0])
    np.testing.assert_allclose(y("none"), [6.0, 0.0])


def test_integer_codes():
    q, scale = D.quantize_i8(np.array([[0.0, 0.0], [254.0, -1.0], [-63.5, 1.25], [1e-3, 5e-4]]))
    assert q.dtype == np.int8 and scale.dtype == np.float32
    assert q[0].tolist() == [0, 0] and scale[0] == np.float32(2.0 ** -100) * (np.float32(1) / np.float32(127))
    assert q[1].tolist() == [127, 0] and scale[1] == 2.0   # -0.5 goes to the even 0
    assert q[2].tolist() == [-127, 2] and scale[2] == 0.5  # 2.5 goes to the even 2
    assert q[3].tolist() == [127, 64]                      # 63.5 goes to the even 64
