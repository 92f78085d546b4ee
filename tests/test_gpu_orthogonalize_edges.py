"""The orthogonalised update at the ends of its arguments' ranges."""
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, say
from test_gpu_dense import TYPES, U, ids
from test_gpu_orthogonalize import update

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (40, 100), (257, 200), (300, 301)])
def test_the_smallest_eps(rows, cols, dt):
    """Beside a norm of zero 2^12 / eps can leave float64's range (eps below 2.3e-305): zeros stay zeros there too, and any
    other matrix, whose norm is 2^-149 at least, has the bits that it has with any eps that is nothing beside its norm."""
    g = torch.stack([update(torch.Generator().manual_seed(i), rows, cols, dt) + 1e-3 for i in range(3)])
    g[1] = 0.0
    want = B.orthogonalize(g, eps=1e-300)
    assert torch.all(want[1] == 0.0) and bool(torch.isfinite(want).all())
    for eps in (3e-305, 2e-305, 1e-307, 5e-324):
        say(f"[orthogonalize] {rows}x{cols} {dt} eps {eps}")
        assert torch.equal(B.orthogonalize(g, eps=eps), want)
        assert torch.all(B.orthogonalize(g[1], eps=eps) == 0.0)


@pytest.mark.parametrize("rows,cols", [(40, 100), (257, 200)])
def test_nan_and_infinity_with_the_smallest_eps(rows, cols):
    g = torch.stack([update(torch.Generator().manual_seed(i), rows, cols, torch.float32) for i in range(3)])
    g[0, 3, 5], g[2, rows - 1, 0] = float("nan"), float("inf")
    y = B.orthogonalize(g, eps=5e-324)
    assert torch.all(torch.isnan(y[0])) and torch.all(torch.isnan(y[2])) and bool(torch.isfinite(y[1]).all())


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(64, 256), (300, 700), (1536, 1536), (2048, 2500)])
def test_repeats_to_the_bit(rows, cols, dt):
    g = update(torch.Generator().manual_seed(rows), rows, cols, dt)
    y = B.orthogonalize(g)
    for _ in range(3):
        assert torch.equal(B.orthogonalize(g), y)


@pytest.mark.parametrize("rows,cols,steps,dt", [
    (1 << 20, 1, 5, torch.float32), (1, 1 << 20, 5, torch.bfloat16), (1 << 20, 130, 3, torch.float16), (300, 1 << 20, 2, torch.bfloat16),
    (16384, 20001, 1, torch.bfloat16), (20001, 16384, 1, torch.float32)], ids=ids)
def test_the_largest_sides(rows, cols, steps, dt):
    """Sides up to 2^20, in norm against the same steps in 64 bits on the device.

    Two planes: 22 bits of each factor, 2^-16 over these steps; one plane (bf16, sides of 256 on): 11 bits, 3 2^-11; and U
    of the output."""
    g = torch.randn(rows, cols, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dt)
    y = B.orthogonalize(g, steps)
    X = g.double()
    X = X / (X.norm() + 1e-7)
    X = X.t().contiguous() if rows > cols else X
    a, b, c = B.NEWTON_SCHULZ
    for _ in range(steps):
        A = X @ X.t()
        X = torch.addmm(X, torch.addmm(A, A, A, beta=b, alpha=c), X, beta=a)
    X = X.t() if rows > cols else X
    err = float((y.double() - X).norm() / X.norm())
    say(f"[orthogonalize] {rows}x{cols} {dt}: {err:.2g}")
    assert err <= U[dt] + (3 * 2.0 ** -11 if dt == torch.bfloat16 and min(rows, cols) >= 256 else 2.0 ** -16)
