"""The gated layer and layers of 8-bit integers at the most columns and rows they take: values that make every output known."""
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

BF16, I8 = torch.bfloat16, torch.int8


def ones(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype, device=DEV)


@pytest.mark.parametrize("dt", [BF16, I8], ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("rows,inner,outer", [(1, 1, 1 << 26), (3, 16, (1 << 26) - 32), (17, 1, (1 << 26) - 31), (40, 16, 1 << 26)])
def test_gated_columns(rows, inner, outer, dt):
    """2^27 rows of w: few rows of x up to the columns that one launch counts, and past them."""
    say(f"[gated] {rows}x{inner}x{outer} {dt}")
    x, w = ones(rows, inner, dtype=dt), ones(2 * outer, inner, dtype=dt)
    w[outer:] = 3
    w[outer - 1], w[-1], w[7] = 2, 5, -1
    scales = (torch.ones(rows, device=DEV), torch.ones(2 * outer, device=DEV)) if dt == I8 else (None, None)
    y = B.gated_linear(x, w, None, "relu", *scales)["y"]
    one = 3.0 * inner * inner
    assert torch.all(y[:, -1] == 10.0 * inner * inner) and torch.all(y[:, 7] == 0.0)
    y[:, -1], y[:, 7] = one, one
    assert float(y.amin()) == one and float(y.amax()) == one


@pytest.mark.parametrize("rows,inner,outer", [(3, 8, 1 << 26), (40, 1, 1 << 25)])
def test_gated_backward_of_many_columns(rows, inner, outer):
    """gate 1, value 2 and gy 1 throughout: gz = (2, 1), each gradient a count of them."""
    say(f"[gated] backward {rows}x{inner}x{outer}")
    x, w, gy = ones(rows, inner), ones(2 * outer, inner), ones(rows, outer)
    z = ones(rows, 2 * outer)
    z[:, outer:] = 2.0
    w[outer:] = -2.0  # gx = sum over the columns of 2 - 2 = 0
    w[5], w[-1] = 9.0, -4.0  # + 16 and - 2
    b = B.gated_linear_backward(gy, x, w, z, "none")
    assert torch.all(b["gx"] == 14.0)
    for k in ("gw", "gbias"):
        assert torch.all(b[k][:outer] == 2.0 * rows) and torch.all(b[k][outer:] == 1.0 * rows)


@pytest.mark.parametrize("rows,outer", [((1 << 30) + 5, 1), ((1 << 31) - 1, 3)])
def test_integer_rows(rows, outer):
    """More rows than one launch counts, each with a scale of its own."""
    say(f"[integers] {rows}x1x{outer}")
    x, w = ones(rows, 1, dtype=I8), ones(outer, 1, dtype=I8)
    xs = torch.full((rows,), 2.0, device=DEV)
    xs[-1], xs[rows // 2] = 5.0, 3.0
    y = B.linear(x, w, x_scale=xs, w_scale=torch.ones(outer, device=DEV))["y"]
    assert torch.all(y[-1] == 5.0) and torch.all(y[rows // 2] == 3.0)
    y[-1], y[rows // 2] = 2.0, 2.0
    assert float(y.amin()) == 2.0 and float(y.amax()) == 2.0


def test_quantised_rows_past_32_bits():
    x = torch.ones((70000, 1), dtype=BF16, device=DEV).expand(70000, 33000).contiguous()
    x[-1, -1] = 127.0
    q = B.quantize_rows(x)
    assert torch.all(q["y"][0] == 127) and torch.all(q["y"][-1, :-1] == 1) and int(q["y"][-1, -1]) == 127
    assert torch.equal(q["scale"][:-1], q["scale"][:1].expand(69999)) and torch.all(q["y"][40000] == 127)
