"""How the binding reads an update's coefficients (CPU only)."""
import numpy as np
import pytest

from equivariant_edge_convolution_amd import binding as B

ONE, TWO = (1.0, 2.0, 3.0), ((1.0, 2.0, 3.0), (4.0, 5.0, 6.0))


def read(coefficients, steps):
    return list(B._coefficients(steps, B._each(coefficients)))


@pytest.mark.parametrize("one", [ONE, list(ONE), (1, 2, 3), np.array(ONE), np.float32(ONE), tuple(np.float32(ONE))])
def test_of_every_step(one):
    assert read(one, 3) == [1.0, 2.0, 3.0] * 3


@pytest.mark.parametrize("each", [TWO, [list(r) for r in TWO], np.array(TWO), np.float32(TWO), tuple(np.float32(TWO))])
def test_of_each_step(each):
    assert read(each, 2) == [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]


@pytest.mark.parametrize("coefficients,steps", [
    ((), 5), ((1.0, 2.0), 5), ((1.0, 2.0, 3.0, 4.0), 5), ((1.0, 2.0, (3.0,)), 3), ((ONE, 4.0), 2), (TWO, 3), (TWO, 1), ((ONE, (1.0, 2.0)), 2),
    (((), ()), 2), (ONE, -1)])
def test_anything_else_is_refused(coefficients, steps):
    with pytest.raises(ValueError, match="coefficients"):
        read(coefficients, steps)
