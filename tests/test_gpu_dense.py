"""The atom-wise dense operators (eec_add_rms_norm, eec_linear and their
backwards) against the float64 oracle, element by element.

Bounds, from the roundings the operators make (U = relative error of one
rounding to the type, EPS = 2^-24 that of float32):
  norm      the sum of squares over at most 64 serial additions per lane and a
            tree: 64 EPS relative, halved by the root; three products: so
            (U + 64 EPS) |y|;
  linear    K additions and K products in any order, each within 2 EPS of the
            running magnitude (a matrix instruction may cut rather than round):
            (2 K + 32) EPS S with S = sum_k |x||w| + |bias|, times the largest
            slope of an activation (1.13) plus 16 EPS of its value and U |y|;
  backward  gz carries U |gz| and 16 EPS |gy| (1 + |z|) from its formula, both
            propagated through sum |gz||w|, then as linear.
Values below the type's normal range are within half of its smallest step.
"""
import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B
from oracle import dense as D

from gpu_util import DEV, np_, say

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "")


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rand(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def view(t, pad, shift=0):
    """The same matrix as columns [shift, shift + width) of a matrix `pad` wider."""
    if pad == 0:
        return t
    raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=raw.dtype, device=t.device)
    wide[:, shift:shift + t.shape[1]] = raw
    out = wide[:, shift:shift + t.shape[1]]
    return out.view(t.dtype) if t.dtype == torch.float8_e4m3fn else out


def within(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.size == 0:
        return
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what  # NaN where the definition has one, and only there
    assert np.all(np.isfinite(got[~np.isnan(ref)])), what
    over = np.where(np.isnan(ref), -np.inf, np.abs(got - ref) - bound)
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}{at}: {got[at]} against {ref[at]}, bound {np.broadcast_to(bound, ref.shape)[at]}"


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (2, 513), (7, 1000), (130, 512), (3, 2047), (2, 4096), (3, 8200), (2, 16400),
               (2, 33001), (0, 64), (600, 96)]


def check_norm(x, weight, residual, out, eps, dt):
    ref = D.norm(f64(x), None if weight is None else f64(weight), None if residual is None else f64(residual), eps)
    if residual is not None:
        within(out["sum"], ref["sum"], (U[dt] + EPS) * np.abs(ref["sum"]) + TINY[dt], "sum")
    within(out["y"], ref["y"], (U[dt] + 64 * EPS) * np.abs(ref["y"]) + TINY[dt], "y")
    within(out["rstd"], ref["rstd"], 64 * EPS * ref["rstd"], "rstd")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,width", NORM_SHAPES)
def test_norm_and_backward(rows, width, dt):
    say(f"[dense] norm {rows}x{width} {dt}")
    g = torch.Generator().manual_seed(rows * 7919 + width)
    for has_res, has_w, pad in ((True, True, 0), (False, True, 3), (True, False, 8)):
        x = view(rand(g, rows, width, dtype=dt), pad, 1 if pad else 0)
        res = view(rand(g, rows, width, dtype=dt), pad) if has_res else None
        w = rand(g, width, dtype=dt) if has_w else None
        out = B.add_rms_norm(x, w, res, eps=1e-5, save_rstd=True)
        check_norm(x, w, res, out, 1e-5, dt)
        gy = view(rand(g, rows, width, dtype=dt), pad)
        gs = rand(g, rows, width, dtype=dt) if has_res else None
        b = B.add_rms_norm_backward(gy, out["sum"], w, out["rstd"], gsum=gs)
        s, rstd, G = f64(out["sum"]), f64(out["rstd"]), f64(gy)
        ref = D.norm_backward(G, s, None if w is None else f64(w), rstd, None if gs is None else f64(gs))
        a = np.abs(G) if w is None else np.abs(G * f64(w))
        xh = np.abs(s) * rstd[:, None]
        # two terms of three products each, and a mean over the row
        size = rstd[:, None] * (a + xh * (a * xh).mean(axis=1, keepdims=True) if rows else a)
        within(b["gx"], ref["gx"], U[dt] * np.abs(ref["gx"]) + 64 * EPS * size + EPS * np.abs(ref["gx"]) + TINY[dt], "gx")
        if w is None:
            assert b["gweight"] is None
        else:
            bound = U[dt] * np.abs(ref["gweight"]) + (rows + 8) * EPS * (np.abs(G) * xh).sum(axis=0) + TINY[dt]
            within(b["gweight"], ref["gweight"], bound, "gweight")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,width", [(1, 1), (4, 65), (3, 512), (5, 1023), (2, 4096), (2, 9000), (2, 33001)])
def test_norm_e4m3(rows, width, dt):
    g = torch.Generator().manual_seed(rows * 31 + width)
    x, res, w = rand(g, rows, width, dtype=dt), rand(g, rows, width, dtype=dt), rand(g, width, dtype=dt)
    out = B.add_rms_norm(x, w, res, quantize=True)
    assert out["y"].dtype == torch.float8_e4m3fn
    y = D.norm(f64(x), f64(w), f64(res), 1e-6)["y"]
    scale = D.e4m3_scale(y)
    within(out["scale"], scale, 64 * EPS * scale, "scale")
    v = y / scale[:, None]
    # half a step of e4m3: 2^-4 of the value, 2^-10 below its normal range; the value itself within 128 EPS
    q = out["y"].cpu().to(torch.float32).numpy().astype(np.float64)
    within(q, v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + 128 * EPS * np.abs(v), "codes")
    assert np.abs(q).max() == 448.0 or rows == 0


def test_norm_empty_and_special_rows():
    x = torch.ones((6, 100), device=DEV)
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1e-30
    x[4, 99] = -float("inf")
    out = B.add_rms_norm(x, None, None, eps=1e-6, save_rstd=True)
    y = np_(out["y"])
    assert np.all(y[0] == 0.0) and np.all(np.isnan(y[1]))
    assert np.isnan(y[2, 5]) and np.all(np.delete(y[2], 5) == 0.0)
    assert np.all(np.isfinite(y[3])) and np.isnan(y[4, 99])
    np.testing.assert_allclose(y[5], 1.0, rtol=1e-5)
    q = B.add_rms_norm(x, None, None, quantize=True)
    scale, codes = np_(q["scale"]), q["y"].float().cpu().numpy()
    assert scale[0] == np.float32(2.0 ** -100) / np.float32(448.0) and np.all(codes[0] == 0.0)
    for bad in (1, 2, 4):
        assert np.isnan(scale[bad]) and np.all(np.isnan(codes[bad]))
    assert np.all(np.abs(codes[5]) == 448.0)
    # eps = 0 and a row of zeros: 0 / 0 by the formula
    assert np.all(np.isnan(np_(B.add_rms_norm(x[:1], eps=0.0)["y"])))


# ------------------------------------------------------------------ linear

LINEAR_SHAPES = [  # rows, inner, outer
    (1, 1, 1), (1, 64, 64), (3, 0, 5), (0, 16, 8), (17, 33, 65), (128, 128, 128), (129, 257, 130), (300, 1029, 7),
    (5, 2050, 300), (1000, 64, 256), (16, 512, 48), (33, 4096, 264), (64, 96, 1000), (257, 320, 513), (2, 8, 4096),
    (512, 1024, 512), (1, 5000, 3)]


def linear_bound(x, w, bias, dt, z, y, inner):
    S = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    ez = (2 * inner + 32) * EPS * S
    return ez + U[dt] * np.abs(z) + TINY[dt], 1.13 * ez + 16 * EPS * (np.abs(z) + np.abs(y)) + U[dt] * np.abs(y) + TINY[dt]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", LINEAR_SHAPES)
def test_linear_and_backward(rows, inner, outer, dt):
    say(f"[dense] linear {rows}x{inner}x{outer} {dt}")
    g = torch.Generator().manual_seed(rows * 7919 + inner * 13 + outer)
    for act, has_b, has_r, pad, shift in (("silu", True, True, 0, 0), ("none", False, False, 0, 0),
                                          ("gelu", True, False, 3, 1), ("relu", False, True, 8, 8)):
        x = view(rand(g, rows, inner, dtype=dt), pad, shift)
        w = view(rand(g, outer, inner, dtype=dt, scale=max(inner, 1) ** -0.5), pad, shift)
        bias = rand(g, outer, dtype=dt) if has_b else None
        res = view(rand(g, rows, outer, dtype=dt), pad, shift) if has_r else None
        out = B.linear(x, w, bias, act, res, save_preact=True)
        X, W = f64(x), f64(w)
        ref = D.linear(X, W, None if bias is None else f64(bias), act, None if res is None else f64(res))
        bz, by = linear_bound(X, W, None if bias is None else f64(bias), dt, ref["preact"], ref["y"], inner)
        within(out["preact"], ref["preact"], bz, f"{act} preact")
        within(out["y"], ref["y"], by, f"{act} y")
        # the same without keeping z
        assert torch.equal(B.linear(x, w, bias, act, res)["y"], out["y"])

        gy = view(rand(g, rows, outer, dtype=dt), pad, shift)
        b = B.linear_backward(gy, x, w, out["preact"] if act != "none" else None, act, bias=True)
        z, G = f64(out["preact"]), f64(gy)
        ref = D.linear_backward(G, X, W, z, act)
        u = U[dt] if act != "none" else 0.0
        ez = (u * np.abs(ref["gz"]) + 16 * EPS * np.abs(G) * (1 + np.abs(z)) + TINY[dt]) if act != "none" else 0 * G
        az = np.abs(ref["gz"]) + ez
        within(b["gx"], ref["gx"], ez @ np.abs(W) + (2 * outer + 32) * EPS * (az @ np.abs(W)) +
               U[dt] * np.abs(ref["gx"]) + TINY[dt], f"{act} gx")
        within(b["gw"], ref["gw"], ez.T @ np.abs(X) + (2 * rows + 32) * EPS * (az.T @ np.abs(X)) +
               U[dt] * np.abs(ref["gw"]) + TINY[dt], f"{act} gw")
        within(b["gbias"], ref["gbias"], (16 * EPS * np.abs(G) * (1 + np.abs(z))).sum(axis=0) +
               (2 * rows + 32) * EPS * az.sum(axis=0) + U[dt] * np.abs(ref["gbias"]) + TINY[dt], f"{act} gbias")


PACKED_SHAPES = [(640, 1100, 601), (700, 901, 777), (1031, 640, 643), (517, 1543, 521), (1301, 1301, 1301), (900, 512, 71),
                 (1751, 1701, 1711)]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", PACKED_SHAPES)
def test_linear_and_backward_packed(rows, inner, outer, dt):
    """Sizes whose operands are packed first (float32 into its parts, odd rows to aligned ones)."""
    test_linear_and_backward(rows, inner, outer, dt)


@pytest.mark.parametrize("rows,inner,outer", [(640, 1100, 601), (1301, 1301, 1301)])
def test_linear_packed_special_values(rows, inner, outer):
    """An infinity or NaN in a packed float32 product reaches its own row alone, also beside values whose parts are zero."""
    x = torch.full((rows, inner), 2.0, device=DEV)
    w = torch.full((outer, inner), 0.5, device=DEV)
    w[3] = -0.5
    x[1, 5], x[2, 7], x[4, 9] = float("inf"), float("nan"), -float("inf")
    x[4, 10], w[5, 9] = float("inf"), 0.0
    y = np_(B.linear(x, w)["y"])
    assert np.all(np.isposinf(np.delete(y[1], 3))) and np.isneginf(y[1, 3])
    assert np.all(np.isnan(y[2])) and np.all(np.isnan(np.delete(y[4], 5))) and np.isnan(y[4, 5])
    rest = np.delete(y, (1, 2, 4), axis=0)
    ref = np.full(outer, float(inner))
    ref[3], ref[5] = -inner, inner - 1
    np.testing.assert_allclose(rest, np.broadcast_to(ref, rest.shape), rtol=2.0 ** -22)


@pytest.mark.parametrize("rows,inner,outer", [(640, 1100, 601), (517, 1543, 521), (300, 4097, 1000), (1301, 1305, 1301),
                                              (1501, 1505, 1503)])
def test_linear_e4m3_packed(rows, inner, outer):
    test_linear_e4m3(rows, inner, outer, torch.bfloat16)


# several workgroups a CU, 256 x 256 tiles; aligned and odd
LARGE_SHAPES = [(2048, 2064, 2080), (2051, 2049, 2050), (2944, 2912, 2960), (2901, 2905, 2899)]


def large_within(got, ref, bound, what):
    """`within` on the device, of finite values."""
    over = (got.double() - ref).abs() - bound
    at = int(torch.argmax(over))
    assert bool(torch.isfinite(got.float()).all()), what
    assert float(over.flatten()[at]) <= 0, f"{what}[{at}]: {float(got.flatten()[at])} against {float(ref.flatten()[at])}"


@pytest.mark.parametrize("dt", TYPES + [torch.float8_e4m3fn], ids=ids)
@pytest.mark.parametrize("rows,inner,outer", LARGE_SHAPES)
def test_linear_large(rows, inner, outer, dt):
    """As the smaller ones, the 64-bit products taken by the library on the device."""
    say(f"[dense] large {rows}x{inner}x{outer} {dt}")
    g = torch.Generator().manual_seed(rows + 3 * inner + 5 * outer)
    eight = dt == torch.float8_e4m3fn
    ot = torch.bfloat16 if eight else dt
    x = rand(g, rows, inner, dtype=dt, scale=30.0 if eight else 1.0)
    w = rand(g, outer, inner, dtype=dt, scale=30.0 if eight else inner ** -0.5)
    xs = rand(g, rows).abs() * 0.01 + 0.001 if eight else None
    ws = (rand(g, outer).abs() * 0.01 + 0.001) * inner ** -0.5 if eight else None
    bias, res = rand(g, outer, dtype=ot), rand(g, rows, outer, dtype=ot)
    out = B.linear(x, w, bias, "silu", res, x_scale=xs, w_scale=ws, out_dtype=ot, save_preact=True)
    X, W = x.float().double(), w.float().double()
    if eight:
        X, W = X * xs.double()[:, None], W * ws.double()[:, None]
    z = X @ W.t() + bias.double()
    y = torch.nn.functional.silu(z) + res.double()
    ez = (2 * inner + 32) * EPS * (X.abs() @ W.abs().t() + bias.double().abs())
    large_within(out["preact"], z, ez + U[ot] * z.abs() + TINY[ot], "preact")
    large_within(out["y"], y, 1.13 * ez + 16 * EPS * (z.abs() + y.abs()) + U[ot] * y.abs() + TINY[ot], "y")
    if eight:
        return
    gy = rand(g, rows, outer, dtype=dt)
    b = B.linear_backward(gy, x, w, out["preact"], "silu", bias=True)
    z, G = out["preact"].double(), gy.double()
    p = torch.sigmoid(z)
    gz = G * p * (1 + z * (1 - p))
    formula = 16 * EPS * G.abs() * (1 + z.abs())
    e = U[dt] * gz.abs() + formula + TINY[dt]
    a = gz.abs() + e
    for what, ref, bound in (
            ("gx", gz @ W, e @ W.abs() + (2 * outer + 32) * EPS * (a @ W.abs())),
            ("gw", gz.t() @ X, e.t() @ X.abs() + (2 * rows + 32) * EPS * (a.t() @ X.abs())),
            ("gbias", gz.sum(dim=0), formula.sum(dim=0) + (2 * rows + 32) * EPS * a.sum(dim=0))):
        large_within(b[what], ref, bound + U[dt] * ref.abs() + TINY[dt], what)


@pytest.mark.parametrize("ot", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", [(1, 64, 64), (3, 16, 5), (17, 1000, 65), (129, 257, 130), (300, 4096, 40),
                                              (256, 512, 512), (1, 4096, 1024), (40, 130, 300), (0, 8, 8), (4, 0, 4)])
def test_linear_e4m3(rows, inner, outer, ot):
    # at 100 a few values lie past e4m3's range and are NaN codes, at 30 none is
    g = torch.Generator().manual_seed(rows * 7 + inner + outer)
    for act, pad, shift, size in (("silu", 0, 0, 100.0), ("none", 5, 3, 100.0), ("gelu", 16, 16, 100.0),
                                  ("silu", 0, 0, 30.0), ("none", 3, 2, 30.0), ("relu", 16, 0, 30.0)):
        x = view(rand(g, rows, inner, scale=size).to(torch.float8_e4m3fn), pad, shift)
        w = view(rand(g, outer, inner, scale=size).to(torch.float8_e4m3fn), pad, shift)
        xs = rand(g, rows).abs() * 0.01 + 0.001
        ws = (rand(g, outer).abs() * 0.01 + 0.001) * max(inner, 1) ** -0.5
        bias, res = rand(g, outer, dtype=ot), rand(g, rows, outer, dtype=ot)
        out = B.linear(x, w, bias, act, res, x_scale=xs, w_scale=ws, out_dtype=ot, save_preact=True)
        X = x.float().cpu().numpy().astype(np.float64) * f64(xs)[:, None]
        W = w.float().cpu().numpy().astype(np.float64) * f64(ws)[:, None]
        ref = D.linear(X, W, f64(bias), act, f64(res))
        bz, by = linear_bound(X, W, f64(bias), ot, ref["preact"], ref["y"], inner)
        within(out["preact"], ref["preact"], bz, f"{act} preact")
        within(out["y"], ref["y"], by, f"{act} y")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", [(3, 40, 24), (200, 256, 256)])
def test_linear_special_values(rows, inner, outer, dt):
    """One infinity or NaN reaches its own row (column) alone, and as the formula has it."""
    g = torch.Generator().manual_seed(3)
    x, w = rand(g, rows, inner, dtype=dt), rand(g, outer, inner, dtype=dt)
    w = torch.where(w.abs() < 0.01, torch.ones_like(w), w)  # no product of an infinity and zero
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    y = np_(B.linear(x, w)["y"].float())
    sign = np.sign(f64(w)[:, 5])
    assert np.array_equal(y[1], np.where(sign > 0, np.inf, -np.inf))
    assert np.all(np.isnan(y[2])) and np.all(np.isfinite(np.delete(y, (1, 2), axis=0)))
    # powers of two: float32's parts below the first are zero
    x = torch.full((rows, inner), 2.0, dtype=dt, device=DEV)
    w = torch.full((outer, inner), 0.5, dtype=dt, device=DEV)
    x[0, 0] = float("inf")
    y = np_(B.linear(x, w)["y"].float())
    assert np.all(np.isposinf(y[0])) and np.all(y[1:] == inner)
    # padding past the end of a row is never read into a sum
    wide = torch.full((rows, inner + 9), float("nan"), dtype=dt, device=DEV)
    wide[:, :inner] = 1.0
    y = np_(B.linear(wide[:, :inner], w)["y"].float())
    assert np.all(y == 0.5 * inner)


def test_linear_float32_keeps_its_accuracy():
    """The error of float32 products is that of float32 arithmetic (2-norm well under 1e-6), large and small inputs alike."""
    g = torch.Generator().manual_seed(5)
    for scale in (1.0, 1e-20, 1e15):
        x, w = rand(g, 256, 1024, scale=scale), rand(g, 192, 1024)
        y = f64(B.linear(x, w)["y"])
        ref = f64(x) @ f64(w).T
        assert np.linalg.norm(y - ref) <= 5e-7 * np.linalg.norm(ref), scale


@pytest.mark.xfail(strict=True, reason="float32 operands are held to 2^-133: 1.2e-38 keeps 8 of its 24 bits")
def test_linear_float32_extremes():
    # largest and smallest magnitudes neither overflow nor vanish
    x = torch.tensor([[3.4e38, 1.2e-38]], device=DEV)
    y = f64(B.linear(x, torch.eye(2, device=DEV))["y"])
    np.testing.assert_allclose(y, f64(x), rtol=2e-7)


def test_linear_float32_extremes_within_the_parts_range():
    v = torch.tensor([[3.4e38, -3.3e38, 1e-32, 3e-33, 1.2e-38, -1e-41, 0.0, -1e30]], device=DEV)
    y = f64(B.linear(v, torch.eye(8, device=DEV))["y"])
    assert np.all(np.abs(y - f64(v)) <= 2e-7 * np.abs(f64(v)) + 3 * 2.0 ** -133)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_gradients_against_differences(dt):
    """The kernels' gradients against central differences of the float64 forward, along random directions."""
    g = torch.Generator().manual_seed(11)
    rows, inner, outer = 9, 31, 18
    x, w, bias, res = (rand(g, rows, inner, dtype=dt), rand(g, outer, inner, dtype=dt, scale=inner ** -0.5),
                       rand(g, outer, dtype=dt), rand(g, rows, inner, dtype=dt))
    gamma, gy = rand(g, inner, dtype=dt), rand(g, rows, outer, dtype=dt)
    n = B.add_rms_norm(x, gamma, res, save_rstd=True)
    f = B.linear(n["y"], w, bias, "silu", save_preact=True)
    bl = B.linear_backward(gy, n["y"], w, f["preact"], "silu")
    bn = B.add_rms_norm_backward(bl["gx"], n["sum"], gamma, n["rstd"])
    loss = lambda x, gamma, w, b: (D.linear(D.norm(x, gamma, f64(res))["y"], w, b, "silu")["y"] * f64(gy)).sum()
    at = [f64(x), f64(gamma), f64(w), f64(bias)]
    grads = [f64(bn["gx"]), f64(bn["gweight"]), f64(bl["gw"]), f64(bl["gbias"])]
    r = np.random.default_rng(0)
    for k, (v, gr) in enumerate(zip(at, grads)):
        d = r.normal(size=v.shape)
        h = 1e-6
        up, dn = list(at), list(at)
        up[k], dn[k] = v + h * d, v - h * d
        num = (loss(*up) - loss(*dn)) / (2 * h)
        # four roundings of intermediate values on the way, in a sum of the gradient's own size
        assert abs(num - (gr * d).sum()) <= 8 * U[dt] * np.linalg.norm(gr) * np.linalg.norm(d) + 1e-6, k


# ------------------------------------------------------------------ calls


def test_results_repeat_and_side_stream():
    g = torch.Generator().manual_seed(4)
    x, w, b, gy = (rand(g, 700, 320, dtype=torch.bfloat16), rand(g, 450, 320, dtype=torch.bfloat16),
                   rand(g, 450, dtype=torch.bfloat16), rand(g, 700, 450, dtype=torch.bfloat16))

    def go():
        n = B.add_rms_norm(x, None, x, save_rstd=True)
        f = B.linear(n["y"], w, b, "gelu", save_preact=True)
        bl = B.linear_backward(gy, n["y"], w, f["preact"], "gelu")
        bn = B.add_rms_norm_backward(bl["gx"], n["sum"], x[0].contiguous(), n["rstd"])
        return [f["y"], bl["gx"], bl["gw"], bl["gbias"], bn["gx"], bn["gweight"]]

    first = go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = go()
    side.synchronize()
    for a, b_ in zip(first, second):
        assert torch.equal(a, b_)


def test_binding_refuses_wrong_tensors():
    x, w = torch.ones((4, 8), device=DEV), torch.ones((6, 8), device=DEV)
    for bad in (lambda: B.linear(x, w.half()), lambda: B.linear(x, w[:, :7]), lambda: B.linear(x, w.cpu()),
                lambda: B.linear(x, torch.ones((8, 6), device=DEV).t()), lambda: B.linear(x, w, act="tanh"),
                lambda: B.linear(x, w, bias=torch.ones(5, device=DEV)), lambda: B.linear(x.double(), w.double()),
                lambda: B.linear(x, w, bias=torch.ones(12, device=DEV)[::2]),
                lambda: B.linear_backward(torch.ones((4, 6), device=DEV), x, w, act="silu"),
                lambda: B.add_rms_norm(x, torch.ones(7, device=DEV)), lambda: B.add_rms_norm(x[0]),
                lambda: B.add_rms_norm(x, residual=x[:3])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.linear(x, w, x_scale=torch.ones(4, device=DEV)), lambda: B.linear(x, w, out_dtype=torch.float16),
                lambda: B.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)),
                lambda: B.add_rms_norm(x, eps=-1.0), lambda: B.linear(x[:1].expand(4, 8), w)):
        with pytest.raises(B.EECError):
            bad()
