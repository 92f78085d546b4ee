"""Sizes and arguments at the limits the header names (CPU only).  Nothing is launched: a call that passes the check
under test is stopped by the next one, an output that overlaps an input."""
import pytest

from test_abi_dense import P, linear, linear_bwd, norm


@pytest.mark.parametrize("call,status", [
    # as many outputs as the header allows, however narrow
    (lambda: linear(rows=1 << 30, outer=1, inner=1, ldx=1, ldw=1, y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: linear(rows=(1 << 31) - 1, outer=1, inner=1, ldx=1, ldw=1, y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: linear(rows=(1 << 31) - 1, outer=32, inner=1, ldx=1, ldw=1, y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: linear(rows=1, outer=1 << 27, inner=1, ldx=1, ldw=1, y=P(2)), "EEC_ERR_ALIAS"),
    (lambda: linear(rows=1 << 20, outer=1 << 16, inner=1, ldx=1, ldw=1, y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: linear_bwd(rows=(1 << 31) - 1, outer=1, inner=1, ldgy=1, ldx=1, ldw=1, gx=P(2)), "EEC_ERR_ALIAS"),
    # and no more
    (lambda: linear(rows=1 << 20, outer=(1 << 16) + 1, inner=1, ldx=1, ldw=1, y=P(1)), "EEC_ERR_SHAPE"),
    (lambda: linear_bwd(rows=1 << 20, outer=8, inner=(1 << 16) + 1, ldgy=8, ldx=1 << 17, ldw=1 << 17), "EEC_ERR_SHAPE"),
    (lambda: linear_bwd(rows=8, outer=1 << 20, inner=(1 << 16) + 1, ldgy=1 << 20, ldx=1 << 17, ldw=1 << 17), "EEC_ERR_SHAPE"),
    # of the products that are asked for
    (lambda: linear_bwd(rows=1 << 20, outer=8, inner=1 << 20, ldgy=8, ldx=1 << 20, ldw=1 << 20, gx=None, gw=P(1)),
     "EEC_ERR_ALIAS"),
    (lambda: linear_bwd(rows=8, outer=1 << 20, inner=1 << 20, ldgy=1 << 20, ldx=1 << 20, ldw=1 << 20, gw=None, gx=P(1)),
     "EEC_ERR_ALIAS"),
    (lambda: linear(rows=1 << 20, outer=8, inner=1 << 20, ldx=1 << 20, ldw=1 << 20, y=P(1)), "EEC_ERR_ALIAS"),
])
def test_products_up_to_the_limit(call, status):
    assert call() == status


@pytest.mark.parametrize("eps,status", [
    (0.0, "EEC_ERR_ALIAS"), (1e-45, "EEC_ERR_ALIAS"), (1e-12, "EEC_ERR_ALIAS"), (3.4e38, "EEC_ERR_ALIAS"),
    # float32 would have 0 or infinity in their place, and a row of zeros NaN in place of zeros
    (1e-46, "EEC_ERR_SHAPE"), (1e-300, "EEC_ERR_SHAPE"), (3.5e38, "EEC_ERR_SHAPE"), (1e300, "EEC_ERR_SHAPE"),
    (float("inf"), "EEC_ERR_SHAPE"), (float("-inf"), "EEC_ERR_SHAPE"), (-1e-300, "EEC_ERR_SHAPE"),
])
def test_eps_within_float32(eps, status):
    assert norm(eps=eps, y=P(1)) == status
