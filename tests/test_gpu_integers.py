"""8-bit integers: rows quantised with a scale each (eec_quantize_rows), and products of such rows (eec_linear with EEC_I8)."""
import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B
from oracle import dense as D

from gpu_util import DEV, np_, say
from test_gpu_dense import EPS, TINY, TYPES, U, f64, ids, rand, view, within

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ rows in 8 bits

WIDTHS = [(1, 1), (3, 7), (5, 64), (2, 513), (7, 1000), (130, 512), (3, 2047), (2, 4096), (3, 8200), (2, 16400), (2, 33001),
          (0, 64), (600, 96), (1031, 257)]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,width", WIDTHS)
def test_quantized_rows(rows, width, dt):
    """Codes and scales are those of the float32 arithmetic that the header states, bit for bit."""
    g = torch.Generator().manual_seed(rows * 7919 + width)
    for pad, size in ((0, 1.0), (3, 1e-4), (8, 300.0)):
        x = view(rand(g, rows, width, dtype=dt, scale=size), pad, 1 if pad else 0)
        out = B.quantize_rows(x, torch.int8)
        assert out["y"].dtype == torch.int8 and out["y"].is_contiguous()
        if rows == 0:
            assert out["y"].shape == (0, width) and out["scale"].shape == (0,)
            continue
        q, scale = D.quantize_i8(x.cpu().float().numpy())
        assert np.array_equal(np_(out["scale"]), scale)
        assert np.array_equal(np_(out["y"]), q)
        # e4m3: half a step of the code around the quotient, 2^-4 of it or 2^-10 below its normal range
        eight = B.quantize_rows(x, E4M3)
        scale = np.maximum(np.abs(x.cpu().float().numpy()).max(axis=1), np.float32(2.0 ** -100)) * (np.float32(1) / np.float32(448))
        assert np.array_equal(np_(eight["scale"]), scale)
        v = f64(x) / scale.astype(np.float64)[:, None]
        within(eight["y"].float(), v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + 2 * EPS * np.abs(v), "e4m3")


def test_quotients_of_every_size():
    """Rows from the smallest to the largest float32, quotients next to the halves between codes among them."""
    r = np.random.default_rng(1)
    rows = []
    for p in list(range(-149, 128, 5)) + [127, -100, -99, -81, -80, -79, -74, -73]:
        amax = np.float32(1.9) * np.float32(2.0) ** np.float32(p) if p > -149 else np.float32(2.0 ** -149)
        scale = np.maximum(amax, np.float32(2.0 ** -100)) * (np.float32(1) / np.float32(127))
        halves = (r.integers(-127, 127, 500) + 0.5).astype(np.float32) * scale
        near = np.nextafter(halves, r.choice([-np.inf, np.inf], 500).astype(np.float32), dtype=np.float32)
        x = np.concatenate([[amax], halves, near, r.uniform(-1, 1, 23).astype(np.float32) * amax]).astype(np.float32)
        rows.append(np.clip(x, -amax, amax))
    x = np.stack(rows)
    out = B.quantize_rows(torch.as_tensor(x).to(DEV))
    q, scale = D.quantize_i8(x)
    assert np.array_equal(np_(out["scale"]), scale) and np.array_equal(np_(out["y"]), q)


@pytest.mark.parametrize("width", [5, 600, 20000])
def test_empty_and_special_rows(width):
    x = torch.ones((6, width), device=DEV)
    x[0] = 0.0
    x[1, 3], x[2, 4], x[4, width - 1] = float("nan"), float("inf"), -float("inf")
    x[3] = 1e-35
    # 1e-35 is 0.0016 of the least scale of integers, 0.0057 of that of e4m3, whose smallest codes are multiples of 2^-9
    for codes, most, small in ((torch.int8, 127, 0.0), (E4M3, 448, 3 * 2.0 ** -9)):
        out = B.quantize_rows(x, codes)
        scale, y, least = np_(out["scale"]), out["y"].float().cpu().numpy(), np.float32(2.0 ** -100) * (np.float32(1) / np.float32(most))
        assert scale[0] == least and np.all(y[0] == 0.0) and scale[3] == least and np.all(y[3] == small)
        for bad in (1, 2, 4):
            assert np.isnan(scale[bad]) and np.all(y[bad] == 0.0 if codes == torch.int8 else np.isnan(y[bad]))
        assert np.all(y[5] == most)


# ------------------------------------------------------------------ products

SHAPES = [  # rows, inner, outer
    (1, 1, 1), (1, 64, 64), (3, 0, 5), (0, 16, 8), (17, 33, 65), (32, 4096, 264), (33, 4096, 264), (128, 128, 128), (129, 257, 130),
    (300, 1029, 7), (5, 2050, 300), (64, 96, 1000), (257, 320, 513), (512, 1024, 512), (1, 5000, 3), (600, 4096, 320),
    (1024, 4096, 2048), (2048, 512, 4096), (1536, 1024, 2816), (1501, 1505, 1503), (4100, 160, 264), (40, 8192, 48),
    (70, 272, 200), (129, 16, 66), (257, 1040, 130), (1000, 1504, 1000), (1531, 1029, 2771)]


def codes(g, *s):
    return torch.randint(-128, 128, s, generator=g, dtype=torch.int8).to(DEV)


def product(x, w):
    """x w^T of integers, exactly: float64 holds every sum."""
    return (x.double() @ w.double().t()).cpu().numpy()


@pytest.mark.parametrize("rows,inner,outer", SHAPES)
def test_sums_are_exact(rows, inner, outer):
    """With scales of one and a float32 output the product is the sum of integers, bit for bit, on every path."""
    say(f"[integers] {rows}x{inner}x{outer}")
    g = torch.Generator().manual_seed(rows * 13 + inner * 7 + outer)
    one = lambda n: torch.ones(n, device=DEV)
    for pad, shift in ((0, 0), (3, 1), (16, 16)):
        x, w = view(codes(g, rows, inner), pad, shift), view(codes(g, outer, inner), pad, shift)
        y = B.linear(x, w, x_scale=one(rows), w_scale=one(outer), out_dtype=torch.float32)["y"]
        ref = product(x, w)
        assert np.abs(ref).max(initial=0.0) < 2 ** 24  # each is a float32 number, and so are its parts over k
        assert np.array_equal(f64(y), ref)


@pytest.mark.parametrize("out_dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", SHAPES)
def test_scaled_products(rows, inner, outer, out_dt):
    """Scales, bias, activation and residual. z: the sum rounded to float32 (in parts over k at most 32 times), two products
    and the bias, 64 EPS of sum |x||w| + |bias| together; then as the layer's other types."""
    g = torch.Generator().manual_seed(rows * 17 + inner * 5 + outer)
    x, w = codes(g, rows, inner), codes(g, outer, inner)
    xs, ws = (0.01 + torch.rand(rows, generator=g)).to(DEV), (0.01 + torch.rand(outer, generator=g)).to(DEV) / max(inner, 1)
    bias, res = rand(g, outer, dtype=out_dt), view(rand(g, rows, outer, dtype=out_dt), 3, 1)
    for act in ("none", "relu", "silu", "gelu"):
        out = B.linear(x, w, bias, act, res, xs, ws, out_dt, save_preact=True)
        scale = np.outer(f64(xs), f64(ws))
        z = product(x, w) * scale + f64(bias)
        y = D.act(z, act) + f64(res)
        ez = 64 * EPS * ((x.double().abs() @ w.double().abs().t()).cpu().numpy() * scale + np.abs(f64(bias)))
        within(out["preact"], z, ez + U[out_dt] * np.abs(z) + TINY[out_dt], f"{act} preact")
        within(out["y"], y, 1.13 * ez + 16 * EPS * (np.abs(z) + np.abs(y)) + U[out_dt] * np.abs(y) + TINY[out_dt], f"{act} y")
        if rows * outer > 1 << 20:
            break


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_longest_sums(rows):
    """inner = 131071 of the largest products: 2^31 - 2^14 of either sign, held in 32 bits and in float32."""
    inner, outer = (1 << 17) - 1, 64
    x = torch.full((rows, inner), -128, dtype=torch.int8, device=DEV)
    w = torch.full((outer, inner), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    one = lambda n: torch.ones(n, device=DEV)
    y = np_(B.linear(x, w, x_scale=one(rows), w_scale=one(outer), out_dtype=torch.float32)["y"])
    assert np.all(np.delete(y, 1, axis=1) == 2.0 ** 31 - 2.0 ** 14)
    within(y[:, 1].astype(np.float64), np.full(rows, -128.0 * 127.0 * inner), 64 * EPS * 128.0 * 127.0 * inner, "negative")


def test_special_scales():
    """Scales of any size; a NaN scale makes its row or column NaN, as the formula has it."""
    x, w = torch.full((40, 64), 2, dtype=torch.int8, device=DEV), torch.full((48, 64), 1, dtype=torch.int8, device=DEV)
    xs, ws = torch.ones(40, device=DEV), torch.ones(48, device=DEV)
    xs[3], ws[5], xs[7], ws[9], xs[8] = float("nan"), 1e-30, 1e-15, 1e-35, 1e35
    y = np_(B.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32)["y"])
    assert np.all(np.isnan(y[3]))
    want = 128.0 * np.outer(np_(xs).astype(np.float64), np_(ws).astype(np.float64))
    rest = np.delete(np.arange(40), 3)
    within(y[rest].astype(np.float64), want[rest], 4 * EPS * np.abs(want[rest]) + 2.0 ** -149, "scales")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_quantised_layer(dt):
    """A layer in 8-bit integers as a program runs it: rows and weights quantised by the library, within what the codes
    leave of the layer in 64 bits: half a step, 2^-1 / 127 of the largest value, of each factor."""
    g = torch.Generator().manual_seed(9)
    x, w, bias = rand(g, 700, 512, dtype=dt), rand(g, 320, 512, dtype=dt, scale=512 ** -0.5), rand(g, 320, dtype=dt)
    qx, qw = B.quantize_rows(x), B.quantize_rows(w)
    y = B.linear(qx["y"], qw["y"], bias, "silu", x_scale=qx["scale"], w_scale=qw["scale"], out_dtype=dt)["y"]
    X, W = f64(x), f64(w)
    ex, ew = (np.abs(v).max(axis=1, keepdims=True) * (0.5 / 127) * (1 + 1e-6) for v in (X, W))
    z = X @ W.T + f64(bias)
    ez = np.abs(X) @ (0 * W + ew).T + (0 * X + ex) @ (np.abs(W) + ew).T + 64 * EPS * (np.abs(X) @ np.abs(W).T + np.abs(f64(bias)))
    out = D.act(z, "silu")
    within(y, out, 1.13 * ez + 16 * EPS * (np.abs(z) + np.abs(out)) + U[dt] * np.abs(out) + TINY[dt], "y")


def test_arguments_of_the_binding():
    x, w, one = torch.zeros((4, 8), dtype=torch.int8, device=DEV), torch.zeros((3, 8), dtype=torch.int8, device=DEV), torch.ones(4, device=DEV)
    for call in (lambda: B.quantize_rows(one[None], torch.float16), lambda: B.quantize_rows(one), lambda: B.quantize_rows(one[None].cpu()),
                 lambda: B.linear(x, w.float(), x_scale=one, w_scale=one[:3])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.quantize_rows(x), lambda: B.linear(x, w), lambda: B.linear_backward(x[:1, :3], x[:1], w, bias=False),
                 lambda: B.linear(x, w, x_scale=one, w_scale=one[:3], out_dtype=torch.int8)):
        with pytest.raises(B.EECError):
            call()
