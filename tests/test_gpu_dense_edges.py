"""The dense operators where values, sizes and arguments are at their limits, against the definitions in 64 bits.

Bounds as in test_gpu_dense.py: U of one rounding to the output's type, EPS = 2^-24 of each float32 operation."""
import numpy as np
import pytest
import torch
from scipy import special

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV
from test_gpu_dense import EPS, TINY, TYPES, U, f64, ids, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ot", TYPES, ids=ids)
@pytest.mark.parametrize("rows,inner,outer", [(3, 64, 24), (70, 130, 50), (200, 256, 256)])
def test_e4m3_scales_of_any_size(rows, inner, outer, ot):
    """Row scales whose product, or whose product with the sum, leaves float32's range where z does not.

    Constant codes, so that every sum over k is exact: what is left are the scales' two products and the output's rounding."""
    for xs, ws, code in ((1e-30, 1e-15, 448.0), (1e-15, 1e-30, 448.0), (1e20, 1e20, 0.0), (1e35, 1e-35, 448.0),
                         (1e-36, 1e36, 416.0), (3e-39, 7.0, 448.0), (0.01, 0.003, 448.0)):
        x = torch.full((rows, inner), code, device=DEV).to(torch.float8_e4m3fn)
        w = torch.full((outer, inner), 1.5, device=DEV).to(torch.float8_e4m3fn)
        sx, sw = torch.full((rows,), xs, device=DEV), torch.full((outer,), ws, device=DEV)
        y = B.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=ot)["y"]
        z = f64(sx)[:, None] * f64(sw)[None, :] * (inner * code * 1.5)
        if ot == torch.float16 and z.max() > 65504.0:
            assert bool(torch.isinf(y).all())
        else:
            within(y, z, (U[ot] + 4 * EPS) * z + TINY[ot], f"{xs} {ws} {code}")


def test_rows_up_to_the_limit():
    """2^31 - 1 rows of one column: one product of as many outputs, and sums over as many rows."""
    rows = 2 ** 31 - 1
    x = torch.empty((rows, 1), dtype=torch.bfloat16, device=DEV)
    x.view(-1)[: rows // 2] = 3.0
    x.view(-1)[rows // 2:] = -5.0
    x[-1] = 7.0
    w, bias = torch.full((1, 1), 2.0, dtype=x.dtype, device=DEV), torch.full((1,), 0.5, dtype=x.dtype, device=DEV)
    y = B.linear(x, w, bias, residual=x)["y"]
    for part in (slice(0, rows // 2), slice(rows // 2, rows - 1), slice(rows - 1, rows)):
        v = float(x[part][0])
        assert bool((y[part] == 3.0 * v + 0.5).all()), part
    del y
    b = B.linear_backward(x, x, w)
    for part in (slice(0, rows // 2), slice(rows // 2, rows - 1), slice(rows - 1, rows)):
        assert bool((b["gx"][part] == 2.0 * float(x[part][0])).all()), part
    # sums of at most 2^22 equal terms are exact in float32; joined in order, then rounded
    gw, gb = 9.0 * (rows // 2) + 25.0 * (rows // 2) + 49.0, -2.0 * (rows // 2) + 7.0
    assert abs(float(b["gw"]) - gw) <= 2.0 ** -7 * gw and abs(float(b["gbias"]) - gb) <= 2.0 ** -7 * abs(gb)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("outer", [2 ** 27 - 16, 2 ** 27])
def test_outputs_up_to_the_limit(outer, rows):
    """The widest layers of one and of a few rows."""
    w = torch.arange(outer, device=DEV, dtype=torch.float32).remainder_(251).to(torch.bfloat16)[:, None]
    x = torch.tensor([1.0, -2.0, 4.0, 0.5] * 5, device=DEV, dtype=w.dtype)[:rows, None]
    y = B.linear(x, w)["y"]
    for i in range(rows):
        assert torch.equal(y[i], w[:, 0] * float(x[i, 0])), i


def test_workspace_of_the_wrong_kind_is_refused():
    x, w = torch.randn(300, 1320, device=DEV), torch.randn(280, 1320, device=DEV)
    gy, rstd = torch.randn(300, 280, device=DEV), torch.ones(300, device=DEV)
    gain = torch.ones(1320, device=DEV)
    calls = (lambda ws: B.linear(x, w, workspace=ws)["y"],
             lambda ws: B.linear_backward(gy, x, w, workspace=ws)["gw"],
             lambda ws: B.add_rms_norm_backward(x, x, gain, rstd, workspace=ws)["gweight"])
    for call in calls:
        size = 16 << 20
        for bad in (torch.empty(size, dtype=torch.uint8), torch.empty(size, dtype=torch.uint8).pin_memory(),
                    torch.empty((2, size), dtype=torch.uint8, device=DEV)[:, ::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        with pytest.raises(B.EECError, match="WORKSPACE"):
            call(torch.empty(256, dtype=torch.uint8, device=DEV))
        # its bytes count, whatever it is made of
        assert torch.equal(call(torch.empty(size // 4, dtype=torch.float32, device=DEV)), call(None))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_backward_without_outputs(act):
    """A layer of no outputs: nothing reaches x, and the other gradients are empty."""
    x, w = torch.ones((4, 8), device=DEV), torch.ones((0, 8), device=DEV)
    out = B.linear(x, w, act=act, save_preact=True)
    b = B.linear_backward(torch.ones((4, 0), device=DEV), x, w, out["preact"], act)
    assert bool((b["gx"] == 0).all()) and b["gw"].shape == (0, 8) and b["gbias"].shape == (0,)


def test_backward_refuses_a_strided_preact():
    x, w = torch.ones((4, 8), device=DEV), torch.ones((6, 8), device=DEV)
    wide = torch.ones((4, 12), device=DEV)
    for bad in (wide[:, :6], wide[:, ::2], torch.ones((6, 4), device=DEV).t()):
        with pytest.raises(ValueError):
            B.linear_backward(torch.ones((4, 6), device=DEV), x, w, bad, "silu")
    # one row, or one column, of any stride is contiguous
    B.linear_backward(torch.ones((1, 6), device=DEV), x[:1], w, wide[:1, :6], "silu")


def act_values(dt, act, n):
    lo = -87.0 if act == "silu" else -13.0  # exp(-|z|), exp(-z^2 / 2) stay normal float32
    return torch.linspace(lo, 9.0, n, dtype=torch.float64).to(dt).to(DEV)[:, None]


def act_bound(dt, act, z):
    """In EPS of the value: the functions 16; with 16-bit outputs the exponential's argument is rounded as well, by 2.5 EPS of
    z^2 / 2 (GELU: the square, the constant, their product) or 1.5 EPS of |z| (SiLU)."""
    if dt == torch.float32:
        return 16.0 + 0 * z
    return 16.0 + (1.5 * np.abs(z) if act == "silu" else 1.25 * z * z)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [32, 4001])
def test_activation_tails(rows, act, dt):
    """A layer of one input and weight 1 is its activation: right to the output's rounding where it is small, too."""
    x, one = act_values(dt, act, rows), torch.ones((1, 1), dtype=dt, device=DEV)
    out = B.linear(x, one, act=act, save_preact=True)
    assert torch.equal(out["preact"], x)
    z = f64(x)
    if act == "silu":
        y = z / (1.0 + np.exp(-z))
    else:
        y = 0.5 * z * special.erfc(-z / np.sqrt(2.0))
    within(out["y"], y, (U[dt] + act_bound(dt, act, z) * EPS) * np.abs(y) + TINY[dt], "y")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_slope_tails(act, dt):
    """Read from gbias: a product would hold float32 slopes to 2^-131 only."""
    z = act_values(dt, act, 4001)
    one = torch.ones((1, 1), dtype=dt, device=DEV)
    slope = B.linear_backward(torch.ones_like(z.t()), one, torch.ones_like(z), z.t().contiguous(), act)["gbias"][:, None]
    v = f64(z)
    if act == "silu":
        p, q = 1.0 / (1.0 + np.exp(-v)), 1.0 / (1.0 + np.exp(v))
        a, b = p, v * p * q
    else:
        a, b = 0.5 * special.erfc(-v / np.sqrt(2.0)), v * np.exp(-0.5 * v * v) / np.sqrt(2.0 * np.pi)
    within(slope, a + b, U[dt] * np.abs(a + b) + act_bound(dt, act, v) * EPS * (np.abs(a) + np.abs(b)) + TINY[dt], "slope")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_activations_of_special_values(dt):
    """As the definitions have them: 0 times infinity is NaN."""
    x = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 30.0, -30.0] * 8, dtype=dt, device=DEV)[:, None]
    one = torch.ones((1, 1), dtype=dt, device=DEV)
    for act, at_minus in (("relu", 0.0), ("silu", float("nan")), ("gelu", float("nan"))):
        y = f64(B.linear(x, one, act=act)["y"])[:7, 0]
        assert y[0] == 0.0 and y[1] == 0.0 and y[2] == np.inf and np.isnan(y[4]) and y[5] == 30.0, act
        assert (np.isnan(y[3]) if np.isnan(at_minus) else y[3] == at_minus) and abs(y[6]) < 1e-11, act


def e4m3_codes(kind, rows, k, g):
    """[rows][k] of e4m3: every code (no NaN), normal values, or groups of eight whose largest product hides the others."""
    if kind == "codes":
        u = torch.randint(0, 254, (rows, k), generator=g, dtype=torch.int64)
        u = torch.where(u >= 127, u + 1, u)  # 0x7f and 0xff are NaN
        return u.to(torch.uint8).view(torch.float8_e4m3fn).to(DEV)
    if kind == "normal":
        return (30.0 * torch.randn(rows, k, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)
    # products 2^16 and, seven times, 1.875 1.875 2^2: just under two steps of 2^3, cut to one each
    v = torch.full((rows, k), 3.75)
    v[:, ::8] = 256.0
    return v.to(torch.float8_e4m3fn).to(DEV)


@pytest.mark.parametrize("ot", [torch.float16, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("kind", ["codes", "normal", "hidden"])
@pytest.mark.parametrize("rows,inner,outer", [(16, 64, 64), (16, 4096, 40), (64, 64, 64), (200, 4096, 256), (300, 8192, 264),
                                              (70, 4095, 50)])
def test_e4m3_sums_with_16_bit_outputs(rows, inner, outer, kind, ot):
    """Within 2^-10 of sum |x||w| whatever the length: 7 2^-13 from the cut products, and from float32's sums of k / 8
    groups 2^-24 each, 2^-14 at k = 8192."""
    g = torch.Generator().manual_seed(inner + rows)
    x, w = e4m3_codes(kind, rows, inner, g), e4m3_codes(kind, outer, inner, g)
    sx, sw = torch.full((rows,), 2.0 ** -8, device=DEV), torch.full((outer,), 2.0 ** -8, device=DEV)
    X, W = x.float().double() * 2.0 ** -8, w.float().double() * 2.0 ** -8
    z, S = f64(X @ W.t()), f64(X.abs() @ W.abs().t())
    y = B.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=ot)["y"]
    within(y, z, 2.0 ** -10 * S + U[ot] * np.abs(z) + TINY[ot], "16-bit output")
    wide = B.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=torch.float32)["y"]
    within(wide, z, (inner / 8 + 32) * EPS * S, "float32 output")


@pytest.mark.parametrize("rows,width,groups", [(1000, 64, 250), (1001, 500, 251), (9, 64, 3), (5000, 64, 512), (100, 4096, 100)])
def test_norm_backward_has_no_group_without_rows(rows, width, groups):
    """The weight gradient's partial rows are those of workgroups that have rows (four at a time where a wave takes one)."""
    g = torch.Generator().manual_seed(rows)
    s, gy = (torch.randn(rows, width, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    w, rstd = torch.ones(width, dtype=torch.bfloat16, device=DEV), torch.ones(rows, device=DEV)
    floats = B.lib().eec_add_rms_norm_backward_workspace_bytes(rows, width) // 4
    ws = torch.full((floats,), -1234.5, device=DEV)
    gw = B.add_rms_norm_backward(gy, s, w, rstd, workspace=ws)["gweight"]
    assert bool((ws[groups * width:] == -1234.5).all()) and bool((ws[: groups * width] != -1234.5).all())
    a, size = f64(gy) * f64(s), np.abs(f64(gy) * f64(s)).sum(axis=0)
    within(gw, a.sum(axis=0), U[torch.bfloat16] * np.abs(a.sum(axis=0)) + (rows + 8) * EPS * size + TINY[torch.bfloat16], "gweight")
