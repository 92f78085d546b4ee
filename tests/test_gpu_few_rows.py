"""Layers of few rows: what is left of k past whole runs of 128 bytes, at every length, type and address.

The operands lie between values that would show in any output: NaN, or codes of 127 (e4m3: NaN)."""
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, np_, say
from test_gpu_dense import EPS, U, f64, ids, within

pytestmark = pytest.mark.gpu

F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


def between(t, before, after):
    """The same rows with `before` and `after` elements of another kind around each."""
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    wide = torch.full((t.shape[0], before + t.shape[1] + after), 0x7f if t.element_size() == 1 else float("nan"), dtype=raw.dtype, device=DEV)
    wide[:, before:before + t.shape[1]] = raw
    return wide[:, before:before + t.shape[1]].view(t.dtype) if t.element_size() == 1 else wide[:, before:before + t.shape[1]]


def operands(g, dt, *shape):
    if dt == I8:
        return torch.randint(-128, 128, shape, generator=g, dtype=I8).to(DEV)
    return torch.randn(*shape, generator=g).to(dt).to(DEV)


@pytest.mark.parametrize("dt,out", [(F32, F32), (F16, F16), (BF16, BF16), (E4M3, BF16), (E4M3, F32), (I8, BF16), (I8, F32)], ids=ids)
@pytest.mark.parametrize("rows", [1, 16, 19])
def test_every_rest(rows, dt, out):
    """z = x w^T within (2 k + 32) EPS sum |x||w| (e4m3 to 16 bits: and 2^-10 of it; integers exactly) and U |z|."""
    g = torch.Generator().manual_seed(rows)
    outer = 24
    one = lambda n: torch.ones(n, device=DEV)
    eight = dt in (I8, E4M3)
    scales = (one(rows), one(outer)) if eight else (None, None)
    lengths = list(range(1, 35)) + [63, 64, 65, 95, 97, 127, 128, 129, 130, 131, 143, 159, 160, 161, 190, 255, 257, 510, 513, 1023, 1025, 1029, 1152,
                                    1153, 2047, 2050, 3199, 4095, 4097, 4100, 5121]
    for k in lengths:
        for before, after in ((0, 0), (0, 3), (1, 2), (4, 12 - k % 4), (2, 1), (3, 5)):
            x, w = between(operands(g, dt, rows, k), before, after), between(operands(g, dt, outer, k), before, after)
            X, W = f64(x.float()), f64(w.float())
            z, S = X @ W.T, abs(X) @ abs(W).T
            e = EPS * S if dt == I8 else ((2 * k + 32) * EPS + (2.0 ** -10 if dt == E4M3 and out != F32 else 0.0)) * S
            y = B.linear(x, w, None, "none", None, *scales, out)["y"]
            within(y, z, e + U[out] * abs(z), f"{k} from {before}")
            h = B.gated_linear(x, w, None, "relu", *scales, out, save_preact=True)["preact"]
            within(h, z, e + U[out] * abs(z), f"gated {k} from {before}")


@pytest.mark.parametrize("dt", [F32, F16, BF16, E4M3, I8], ids=ids)
def test_rest_at_the_end_of_memory(dt):
    """Rows that end where their allocation does, at lengths that are no multiple of a dword, and a k of one."""
    g = torch.Generator().manual_seed(1)
    for rows, k, outer in ((1, 1, 1), (1, 3, 1), (2, 1, 5), (3, 129, 2), (17, 511, 3), (32, 1, 17)):
        x, w = operands(g, dt, rows, k), operands(g, dt, outer, k)
        scales = (torch.ones(rows, device=DEV), torch.ones(outer, device=DEV)) if dt in (I8, E4M3) else (None, None)
        out = F32 if dt in (I8, E4M3) else dt
        y = B.linear(x, w, None, "none", None, *scales, out)["y"]
        X, W = f64(x.float()), f64(w.float())
        within(y, X @ W.T, (2 * k + 32) * EPS * (abs(X) @ abs(W).T) + U[out] * abs(X @ W.T), f"{rows}x{k}x{outer}")
        say(f"[few rows] {rows}x{k}x{outer} {dt}")
