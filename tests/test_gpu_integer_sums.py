"""Layers of 8-bit integers whose sums float32 cannot hold: summed exactly in 32 bits on every path, and rounded once."""
import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, np_, say
from test_gpu_dense import view
from test_gpu_integers import codes

pytestmark = pytest.mark.gpu


def large_codes(g, rows, n):
    """Codes of 64 to 127 with some others between: sums of 9000 a term, above 2^24 from 2000 terms on, odd ones among them."""
    q = torch.randint(64, 128, (rows, n), generator=g, dtype=torch.int8)
    some = torch.rand(rows, n, generator=g) < 0.1
    return torch.where(some, torch.randint(-128, 128, (rows, n), generator=g, dtype=torch.int8), q).to(DEV)


def rounded_sums(x, w):
    """x w^T, exactly (float64 holds every sum), rounded once to float32."""
    z = (x.double() @ w.double().t()).cpu().numpy()
    return z, z.astype(np.float32)


# rows, inner, outer: few rows; split over k in 64, 128 and 256 tiles, aligned, by whole cache lines or not, and packed
SHAPES = [(1, 4096, 64), (17, 8192, 300), (32, 70001, 40), (64, 4096, 512), (33, 4096, 264), (600, 4096, 320), (70, 4097, 300), (500, 4099, 33),
          (600, 8001, 700), (1024, 4096, 1024), (2304, 16384, 2304), (130, 131071, 70)]


@pytest.mark.parametrize("rows,inner,outer", SHAPES)
def test_sums_are_rounded_once(rows, inner, outer):
    say(f"[integer sums] {rows}x{inner}x{outer}")
    g = torch.Generator().manual_seed(rows + inner + outer)
    one = lambda n: torch.ones(n, device=DEV)
    for pad, shift in ((0, 0), (3, 1)):
        x, w = view(large_codes(g, rows, inner), pad, shift), view(large_codes(g, outer, inner), pad, shift)
        exact, want = rounded_sums(x, w)
        assert np.mean(exact != want) > 0.2  # what two roundings would tell from one
        y = np_(B.linear(x, w, x_scale=one(rows), w_scale=one(outer), out_dtype=torch.float32)["y"])
        assert np.array_equal(y, want)
        if rows * outer > 1 << 20:
            break


@pytest.mark.parametrize("rows,inner,outer", [(9, 4096, 64), (64, 4096, 256), (33, 4099, 132), (600, 4096, 161), (600, 8001, 350), (2304, 16384, 1152)])
def test_gated_sums_are_rounded_once(rows, inner, outer):
    say(f"[integer sums] gated {rows}x{inner}x{outer}")
    g = torch.Generator().manual_seed(rows + inner + outer)
    one = lambda n: torch.ones(n, device=DEV)
    x, w = large_codes(g, rows, inner), large_codes(g, 2 * outer, inner)
    exact, want = rounded_sums(x, w)
    assert np.mean(exact != want) > 0.2
    out = B.gated_linear(x, w, None, "relu", one(rows), one(2 * outer), torch.float32, save_preact=True)
    assert np.array_equal(np_(out["preact"]), want)
    gate, value = want[:, :outer], want[:, outer:]
    assert np.array_equal(np_(out["y"]), np.maximum(gate, np.float32(0)) * value)


def test_a_row_does_not_depend_on_the_others():
    """One token alone, in a few, in many: how the sum over k is split goes by their number, its value does not."""
    g = torch.Generator().manual_seed(3)
    x, w = large_codes(g, 3000, 4096), large_codes(g, 264, 4096)
    xs, ws = (0.01 + torch.rand(3000, generator=g)).to(DEV), (0.01 + torch.rand(264, generator=g)).to(DEV)
    bias = torch.randn(264, generator=g).to(DEV)
    layer = lambda n: B.linear(x[:n], w, bias, "silu", x_scale=xs[:n], w_scale=ws, out_dtype=torch.float32)["y"]
    gated = lambda n: B.gated_linear(x[:n], w, bias, "silu", xs[:n], ws, torch.float32)["y"]
    for f in (layer, gated):
        y = f(3000)
        for n in (1, 5, 20, 33, 100, 400, 1100):
            assert torch.equal(f(n), y[:n]), n
