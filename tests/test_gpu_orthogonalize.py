"""The orthogonalised update (eec_orthogonalize) against the float64 oracle, in norm.

Bound: the arithmetic that the kernels are documented to do, done in numpy -- X, A and B held 2^12 times their value in
float16 planes (X in two; the products' operands in one for large bfloat16 updates, in two otherwise, without the product of
the two low parts), sums in float32 -- is off the oracle by what these roundings are worth for this input. The kernels round at
the same places, but sum in another order, so a rounding may fall the other way: three times that, and for inputs so small
that this simulation happens to be exact 2^-10 (one plane: one rounding to 11 bits, twice over) or 2^-20 (two) of the norm; then U, half a step of the type, for the output.
"""
import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B
from oracle import dense as D

from gpu_util import DEV, np_, say
from test_gpu_dense import TYPES, U, f64, ids

pytestmark = pytest.mark.gpu

QUINTIC = (D.QUINTIC,) * 5


def planes(v, two):
    hi = (v * np.float32(4096)).astype(np.float16)
    lo = (v * np.float32(4096) - hi.astype(np.float32)).astype(np.float16) if two else np.zeros_like(hi)
    return hi.astype(np.float32) / np.float32(4096), lo.astype(np.float32) / np.float32(4096)


def simulated(g, coefficients, eps, two):
    """The documented arithmetic; float32 sums."""
    x = (g / (np.sqrt((g * g).sum()) + eps)).astype(np.float32)
    tall = x.shape[0] > x.shape[1]
    x = np.ascontiguousarray(x.T) if tall else x
    mul = lambda p, q: p[0] @ q[0] + (p[0] @ q[1] + p[1] @ q[0] if two else 0)
    for a, b, c in coefficients:
        hi, lo = planes(x, True)
        xs = (hi, lo if two else 0 * lo)
        gram = planes(mul(xs, (xs[0].T, xs[1].T)), two)
        poly = planes(np.float32(b) * (gram[0] + gram[1]) + np.float32(c) * mul(gram, gram), two)
        x = np.float32(a) * (hi + lo) + mul(poly, xs)
    return x.T if tall else x


def off(got, ref):
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)


def check(y, g, dt, coefficients=QUINTIC, eps=1e-7, what=""):
    G = f64(g)
    ref, two = D.orthogonalize(G, coefficients, eps), dt != torch.bfloat16 or min(G.shape) < 256
    least = 2.0 ** -20 if two else 2.0 ** -10
    bound = 3 * off(simulated(G, coefficients, eps, two).astype(np.float64), ref) + least + U[dt]
    err = off(f64(y), ref)
    say(f"[orthogonalize] {what} {list(g.shape)} {dt}: {err:.2g}, bound {bound:.2g}")
    assert err <= bound


def update(g, m, n, dt, spread=0.5):
    """A gradient: a few strong directions over noise that differs from row to row and column to column."""
    r = max(1, min(m, n) // 16)
    u = torch.randn(m, n, generator=g) * torch.exp(spread * torch.randn(m, 1, generator=g)) * torch.exp(spread * torch.randn(1, n, generator=g))
    u += torch.randn(m, r, generator=g) @ torch.randn(r, n, generator=g) * (4 / r ** 0.5)
    return (1e-3 * u).to(dt).to(DEV)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 3), (5, 64), (64, 5), (33, 65), (64, 64), (65, 33), (128, 128), (129, 129), (130, 257), (257, 130),
          (300, 1029), (1029, 300), (512, 512), (16, 3001), (3001, 16), (640, 1000)]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_updates(rows, cols, dt):
    g = update(torch.Generator().manual_seed(rows * 7919 + cols), rows, cols, dt)
    check(B.orthogonalize(g), g, dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("batch,rows,cols", [(1, 1300, 2100), (1, 1536, 1536), (1, 1700, 2100), (1, 2100, 1701), (3, 1290, 1000), (3, 1000, 1290)])
def test_large_updates(batch, rows, cols, dt):
    """Small and large tiles of every kind, above and across the diagonal."""
    gen = torch.Generator().manual_seed(rows)
    g = torch.stack([update(gen, rows, cols, dt) for _ in range(batch)])
    y = B.orthogonalize(g)
    check(y[-1], g[-1], dt)
    if batch > 1:
        check(y[0], g[0], dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("batch,rows,cols", [(1, 53, 5616), (1, 9000, 16), (2, 200, 6001), (1, 260, 20001), (1, 20001, 260), (1, 1, 70000), (70, 20, 300)])
def test_long_updates(batch, rows, cols, dt):
    """Few tiles of long sums, which are split and joined; many small matrices."""
    gen = torch.Generator().manual_seed(rows)
    g = torch.stack([update(gen, rows, cols, dt) for _ in range(batch)])
    y = B.orthogonalize(g)
    check(y[-1], g[-1], dt)
    assert torch.equal(B.orthogonalize(g[0]), y[0]) or batch > 1  # how a sum is split goes by the batch
    check(y[0], g[0], dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_normal_and_steep_updates(dt):
    """Singular values close together, and over many decades."""
    g = torch.Generator().manual_seed(3)
    flat = torch.randn(200, 520, generator=g).to(dt).to(DEV)
    check(B.orthogonalize(flat), flat, dt, what="normal")
    u, s, v = torch.linalg.svd(torch.randn(96, 300, generator=g), full_matrices=False)
    steep = (u * torch.exp(-8 * torch.arange(96) / 96) @ v).to(dt).to(DEV)
    check(B.orthogonalize(steep), steep, dt, what="steep")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(64, 256), (200, 72), (300, 301)])
def test_batches_and_strides(rows, cols, dt):
    """Matrices of a batch are treated one by one, wherever they lie; an only one without a batch alike, bit for bit."""
    gen = torch.Generator().manual_seed(rows)
    wide = torch.zeros((5, rows + 3, cols + 5), dtype=dt, device=DEV)
    g = wide[1:4, 2:2 + rows, 1:1 + cols]
    for i in range(3):
        g[i] = update(gen, rows, cols, dt) * 10.0 ** i
    before = wide.clone()
    y = B.orthogonalize(g)
    assert y.shape == g.shape and y.is_contiguous() and torch.equal(wide, before)
    for i in range(3):
        check(y[i], g[i], dt, what=f"batch {i}")
        assert torch.equal(B.orthogonalize(g[i].contiguous()), y[i]) and torch.equal(B.orthogonalize(g[i]), y[i])
    assert torch.equal(B.orthogonalize(g), y)
    # matrices that interleave, and one several times
    between = torch.stack([g[i] for i in range(3)], dim=1).transpose(0, 1)
    assert between.stride(0) < between.stride(1) and torch.equal(B.orthogonalize(between), y)
    assert torch.equal(B.orthogonalize(g[1].expand(3, rows, cols)), y[1].expand(3, rows, cols))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(40, 100), (257, 200)])
def test_zeros_and_special_values(rows, cols, dt):
    """A matrix of zeros stays one; a NaN or an infinity fills its own matrix with NaN and no other."""
    gen = torch.Generator().manual_seed(1)
    g = torch.stack([update(gen, rows, cols, dt) for _ in range(5)])
    g[1] = 0.0
    g[2, 3, 5], g[3, rows - 1, cols - 1] = float("nan"), float("inf")
    y = B.orthogonalize(g)
    assert torch.all(y[1] == 0.0) and torch.all(torch.isnan(y[2])) and torch.all(torch.isnan(y[3]))
    for i in (0, 4):
        assert torch.equal(y[i], B.orthogonalize(g[i]))
    y = B.orthogonalize(g.transpose(1, 2).contiguous())
    assert torch.all(y[1] == 0.0) and torch.all(torch.isnan(y[2])) and torch.all(torch.isnan(y[3])) and torch.all(torch.isfinite(y[4]))


@pytest.mark.parametrize("dt,powers", [(torch.float32, (-120, -60, 60, 120)), (torch.bfloat16, (-100, 100)), (torch.float16, (-6, 4))], ids=ids)
def test_size_of_the_update_does_not_matter(dt, powers):
    """g times a power of two gives the same bits, squares beyond float32's range included (eps far below any norm)."""
    gen = torch.Generator().manual_seed(2)
    g = (torch.randn(70, 90, generator=gen) + 3.0 * torch.randn(70, 1, generator=gen).sign()).to(dt).to(DEV)  # no value is small beside the others
    y = B.orthogonalize(g, eps=1e-300)
    for p in powers:
        assert torch.equal(B.orthogonalize((g.double() * 2.0 ** p).to(dt), eps=1e-300), y)


def test_eps_beside_the_norm():
    """Norms below eps: X = g / (|g| + eps) is small, and so is what comes of it."""
    g = torch.randn(30, 50, generator=torch.Generator().manual_seed(4)).to(DEV)
    for size, eps in ((1e-9, 1e-7), (1.0, 100.0)):
        check(B.orthogonalize(g * size, eps=eps), g * size, torch.float32, eps=eps, what=f"eps {eps}")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_coefficients(dt):
    """Any number of steps and any coefficients; (1, 0, 0) gives X itself: to 2^-22 of each value, or 2^-37, then rounded."""
    gen = torch.Generator().manual_seed(6)
    for rows, cols in ((48, 80), (80, 48), (200, 150)):
        g = update(gen, rows, cols, dt)
        for coefficients in ((D.QUINTIC,), ((8.28, -23.6, 17.3), (4.1, -2.95, 0.55)), ((2.0, -1.5, 0.5),) * 8):
            check(B.orthogonalize(g, len(coefficients), coefficients), g, dt, coefficients, what=f"{len(coefficients)} steps")
            assert torch.equal(B.orthogonalize(g, len(coefficients), [list(c) for c in coefficients]),
                               B.orthogonalize(g, len(coefficients), coefficients))
        x = f64(g) / (np.linalg.norm(f64(g)) + 1e-7)
        y = f64(B.orthogonalize(g, 1, (1.0, 0.0, 0.0)))
        tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
        assert np.all(np.abs(y - x) <= (U[dt] + 2.0 ** -22) * np.abs(x) + 2.0 ** -37 + tiny)


def test_reaches_orthonormal_rows():
    """Convergent coefficients: rows (columns) orthonormal to float32, singular vectors those of g."""
    g = torch.randn(100, 260, generator=torch.Generator().manual_seed(7))
    u, _, v = torch.linalg.svd(g.double(), full_matrices=False)
    for G, ref in ((g, u @ v), (g.t().contiguous(), (u @ v).t())):
        y = B.orthogonalize(G.to(DEV), 25, (1.875, -1.25, 0.375)).cpu().double()
        assert float((y - ref).norm() / ref.norm()) < 1e-5


def test_side_stream_and_workspace():
    g = update(torch.Generator().manual_seed(8), 150, 333, torch.float32)
    y = B.orthogonalize(g)
    size = B.lib().eec_orthogonalize_workspace_bytes(1, 150, 333, 0)
    ws = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device=DEV)  # NaN wherever something is read before it is written
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = B.orthogonalize(g, workspace=ws[:size])
    side.synchronize()
    assert torch.equal(y, z) and torch.all(ws[size:] == 0xff)


@pytest.mark.parametrize("shape,dt", [((2, 64, 100), torch.float32), ((300, 200), torch.bfloat16)])
def test_in_a_graph(shape, dt):
    """Captured once, replayed with other inputs and eager work in between: every replay equals the eager call."""
    gen = torch.Generator().manual_seed(9)
    fresh = lambda: torch.randn(*shape, generator=gen).to(dt).to(DEV)
    g = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.orthogonalize(g)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = B.orthogonalize(g)
    for _ in range(3):
        g.copy_(fresh())
        eager = B.orthogonalize(g)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_arguments_of_the_binding():
    g = torch.zeros((6, 8), device=DEV)
    for call in (lambda: B.orthogonalize(g[0]), lambda: B.orthogonalize(g.cpu()), lambda: B.orthogonalize(g.t()), lambda: B.orthogonalize(g.double()),
                 lambda: B.orthogonalize(g, 5, ((1.0, 0.0, 0.0),)), lambda: B.orthogonalize(g, 2, ((1.0, 0.0), (1.0, 0.0))),
                 lambda: B.orthogonalize(g, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.orthogonalize(g, 0), lambda: B.orthogonalize(g, eps=0.0), lambda: B.orthogonalize(g, 3, (2.0, 0.0, 0.0)),
                 lambda: B.orthogonalize(torch.zeros((300, 300), device=DEV), workspace=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(B.EECError):
            call()
    assert B.orthogonalize(g[:0]).shape == (0, 8) and B.orthogonalize(g[:, :0]).shape == (6, 0) and B.orthogonalize(g[None][:0]).shape == (0, 6, 8)
