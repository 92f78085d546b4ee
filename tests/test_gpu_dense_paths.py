"""The dense layer's paths, each at sizes that take it (by the workspace it asks for), against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import test_gpu_dense as T
from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, np_

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
SIZE = {torch.float32: 6, torch.float16: 2, torch.bfloat16: 2, E4M3: 1}  # bytes of a packed element


def packed(dt, *shapes):
    return sum(SIZE[dt] * a * b for a, b in shapes)


def forward_bytes(rows, outer, inner, dt):
    out = torch.bfloat16 if dt == E4M3 else dt
    return B.lib().eec_linear_workspace_bytes(rows, outer, inner, B.DTYPES[dt], B.DTYPES[out])


def backward_bytes(rows, outer, inner, dt, act="none"):
    return B.lib().eec_linear_backward_workspace_bytes(rows, outer, inner, B.DTYPES[dt], B.ACTS[act])


@pytest.mark.parametrize("dt,rows,inner,outer", [
    (torch.bfloat16, 1751, 1701, 1711), (torch.float16, 1751, 1701, 1711), (torch.bfloat16, 2900, 1030, 1699),
    (E4M3, 1501, 1505, 1503), (E4M3, 1441, 1450, 1459), (E4M3, 2900, 1030, 1699)], ids=T.ids)
def test_packed_forward(dt, rows, inner, outer):
    """Rows that 16-byte loads do not take are laid out for them first."""
    assert forward_bytes(rows, outer, inner, dt) >= packed(dt, (rows, inner), (outer, inner))
    T.test_linear_large(rows, inner, outer, dt)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=T.ids)
@pytest.mark.parametrize("rows,inner,outer", [(1031, 1037, 1043), (2000, 1001, 520), (2000, 520, 1001)])
def test_packed_backward(rows, inner, outer, dt):
    """x and w, gz, or both laid out first, as inner and outer are odd."""
    shapes = ([(rows, inner), (outer, inner)] if inner % 8 else []) + ([(rows, outer)] if outer % 8 else [])
    assert backward_bytes(rows, outer, inner, dt, "silu") >= packed(dt, *shapes)
    T.test_linear_large(rows, inner, outer, dt)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=T.ids)
@pytest.mark.parametrize("rows,inner,outer", [(4096, 512, 512), (4100, 128, 264), (8211, 256, 136), (5003, 520, 507), (32768, 64, 64)])
def test_weight_gradient_split_over_rows(rows, inner, outer, dt):
    """gw of many rows and few outputs: its sum over the rows is split, and the parts are added in order."""
    assert backward_bytes(rows, outer, inner, dt) >= 2 * 4 * outer * inner
    T.test_linear_large(rows, inner, outer, dt)


@pytest.mark.parametrize("dt,rows,inner,outer", [
    (torch.float32, 1301, 1301, 1301), (torch.float32, 8195, 517, 515), (torch.bfloat16, 1751, 1701, 1711),
    (torch.float16, 1751, 1701, 1711)], ids=T.ids)
def test_special_values_packed(dt, rows, inner, outer):
    """An infinity or a NaN reaches its own row, or column, and no other, beside values whose lower parts are zero."""
    assert forward_bytes(rows, outer, inner, dt) >= packed(dt, (rows, inner), (outer, inner))
    x = torch.full((rows, inner), 2.0, dtype=dt, device=DEV)
    w = torch.full((outer, inner), 0.5, dtype=dt, device=DEV)
    w[3] = -0.5
    x[1, 5], x[2, 7], x[rows - 1, inner - 1] = float("inf"), float("nan"), -float("inf")
    y = np_(B.linear(x, w)["y"].float())
    assert np.all(np.isposinf(np.delete(y[1], 3))) and np.isneginf(y[1, 3])
    assert np.all(np.isneginf(np.delete(y[-1], 3))) and np.isposinf(y[-1, 3])
    assert np.all(np.isnan(y[2]))
    rest = np.delete(y, (1, 2, rows - 1), axis=0)
    ref = np.full(outer, float(inner))
    ref[3] = -inner
    np.testing.assert_allclose(rest, np.broadcast_to(ref, rest.shape), rtol=2.0 ** -22 + T.U[dt])

    gy = torch.full((rows, outer), 0.25, dtype=dt, device=DEV)
    x = torch.full((rows, inner), 2.0, dtype=dt, device=DEV)
    gy[4, 6], gy[7, outer - 1] = float("inf"), float("nan")
    assert backward_bytes(rows, outer, inner, dt) >= packed(dt, (rows, inner), (outer, inner), (rows, outer))
    b = B.linear_backward(gy, x, w)
    gx, gw, gb = (np_(b[k].float()) for k in ("gx", "gw", "gbias"))
    assert np.all(np.isposinf(gx[4])) and np.all(np.isnan(gx[7])) and np.all(np.isfinite(np.delete(gx, (4, 7), axis=0)))
    assert np.all(np.isposinf(gw[6])) and np.all(np.isnan(gw[-1])) and np.all(np.isfinite(np.delete(gw, (6, outer - 1), axis=0)))
    assert np.isposinf(gb[6]) and np.isnan(gb[-1]) and np.all(np.isfinite(np.delete(gb, (6, outer - 1))))
    np.testing.assert_allclose(np.delete(gx, (4, 7), axis=0), 0.125 * (outer - 2), rtol=2.0 ** -22 + T.U[dt])
    np.testing.assert_allclose(np.delete(gw, (6, outer - 1), axis=0), 0.5 * rows, rtol=2.0 ** -22 + T.U[dt])


@pytest.mark.parametrize("rows,inner,outer", [(600001, 8, 1), (600001, 24, 33), (600001, 64, 5)])
def test_backward_of_many_narrow_rows(rows, inner, outer):
    """The workspace stays in proportion to the operands: gz is not padded to rows that dwarf them."""
    assert backward_bytes(rows, outer, inner, torch.bfloat16, "silu") <= 4 * packed(torch.bfloat16, (rows, inner), (rows, outer))
    assert backward_bytes(2 ** 31 - 1, 1, 8, torch.bfloat16, "silu") <= 2 ** 33
    T.test_linear_large(rows, inner, outer, torch.bfloat16)
