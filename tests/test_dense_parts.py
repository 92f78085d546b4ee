"""float32 products in bf16 parts: six of the nine part products, at float32's accuracy.

The operands' three parts are truncated, so what the three products left out are worth has the sign of the whole: with
|m| < 2^-7 and |l| < 2^-15 of a value's power of two at most 2 2^-22 + 2^-30 of each product.

The bound in norm, for values of random sign: a sum over k takes n = 6 k / 32 matrix instructions, each of which rounds
the running sum (by 2^-24 of it at most); the running sums grow like a walk, and so do their roundings, to
2^-24 sqrt(n / 2) of the result; 2 2^-24 stand for the products left out and the last rounding.
"""
import numpy as np
import pytest
import torch

EPS = 2.0 ** -24
LEFT_OUT = 2.0 ** -21 + 2.0 ** -30
TAKEN = ((2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0))  # parts h, m, l of one operand and of the other


def norm_bound(k):
    return EPS * (np.sqrt(6 * k / 64) + 2)


def parts(x):
    """The three truncated bf16 parts of float32 values, as float64."""
    out, rest = [], x.astype(np.float32)
    for _ in range(3):
        h = (rest.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
        out.append(h.astype(np.float64))
        rest = rest - h  # exact
    assert not rest.any()
    return out


def product(x, w, taken=TAKEN):
    X, W = parts(x), parts(w)
    return sum(X[i] @ W[j].T for i, j in taken)


def relative(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("k", [300, 512, 2049, 8192])
def test_the_bound_tells_a_missing_part(k):
    """Six products are well within the bound; without any one of them, or with a part of another row or plane, it fails."""
    r = np.random.default_rng(k)
    x, w = (r.standard_normal((40, k)).astype(np.float32) for _ in range(2))
    ref = x.astype(np.float64) @ w.astype(np.float64).T
    assert relative(product(x, w), ref) < 2 * EPS
    for gone in TAKEN:
        assert relative(product(x, w, [t for t in TAKEN if t != gone]), ref) > 2 * norm_bound(k), gone
    X, W = parts(x), parts(w)
    for part in range(1, 3):
        for wrong in (np.roll(X[part], 1, axis=0), np.roll(X[part], 1, axis=1), X[3 - part], 0 * X[part]):
            Y = list(X)
            Y[part] = wrong
            assert relative(sum(Y[i] @ W[j].T for i, j in TAKEN), ref) > 2 * norm_bound(k), part


def test_what_is_left_out():
    """At most 2^-21 of a product, towards zero; 0.6 x 2^-24 on average over independent values."""
    worst = np.float32(1 + 2.0 ** -7 - 2.0 ** -23)
    v = np.concatenate([np.random.default_rng(0).uniform(1, 2, 100000).astype(np.float32), [worst]])
    for a, b, independent in ((v, v, False), (v, v[::-1].copy(), True)):
        A, B_ = parts(a), parts(b)
        exact = a.astype(np.float64) * b
        off = (exact - sum(A[i] * B_[j] for i, j in TAKEN)) / exact
        assert np.all(off >= 0) and off.max() <= LEFT_OUT
        assert not independent or 0.5 * EPS < off.mean() < 0.8 * EPS
    X = worst.astype(np.float64) ** 2
    assert (X - float(product(worst[None, None], worst[None, None])[0, 0])) / X > 7.5 * EPS


# ------------------------------------------------------------------ on the device


def device_norm(a, b):
    return float((a.double() - b).norm() / b.norm())


def packed_bytes(*shapes):
    """Bytes of float32 operands in three planes, without their padding."""
    return sum(6 * a * b for a, b in shapes)


# rows, inner, outer: what each of them reaches in parts, packed: a whole product, gw split over k, both ragged
SHAPES = [(2051, 2049, 2050), (1301, 1301, 1301), (8192, 512, 512), (8199, 517, 515), (32768, 512, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", SHAPES)
def test_packed_products_keep_float32(rows, inner, outer):
    from equivariant_edge_convolution_amd import binding as B

    assert B.lib().eec_linear_workspace_bytes(rows, outer, inner, 0, 0) >= packed_bytes((rows, inner), (outer, inner))
    assert B.lib().eec_linear_backward_workspace_bytes(rows, outer, inner, 0, 0) >= \
        packed_bytes((rows, inner), (outer, inner), (rows, outer))
    g = torch.Generator().manual_seed(rows + inner)
    x, w, gy = (torch.randn(*s, generator=g).cuda() for s in ((rows, inner), (outer, inner), (rows, outer)))
    X, W, G = x.double(), w.double(), gy.double()
    y = B.linear(x, w)["y"]
    assert device_norm(y, X @ W.t()) <= norm_bound(inner)
    b = B.linear_backward(gy, x, w)
    assert device_norm(b["gx"], G @ W) <= norm_bound(outer)
    assert device_norm(b["gw"], G.t() @ X) <= norm_bound(rows)
    # through an activation, whose gradient is split into its parts where it is computed
    b = B.linear_backward(gy, x, w, y, "relu")
    Z = torch.where(y > 0, G, torch.zeros_like(G))
    assert device_norm(b["gx"], Z @ W) <= norm_bound(outer)
    assert device_norm(b["gw"], Z.t() @ X) <= norm_bound(rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", [(20, 2049, 300), (300, 2049, 300), (1000, 64, 256), (4096, 512, 1)])
def test_other_products_keep_float32(rows, inner, outer):
    """The kernel of few rows, and the general one in both its tile sizes."""
    from equivariant_edge_convolution_amd import binding as B

    g = torch.Generator().manual_seed(rows + inner)
    x, w, gy = (torch.randn(*s, generator=g).cuda() for s in ((rows, inner), (outer, inner), (rows, outer)))
    X, W, G = x.double(), w.double(), gy.double()
    assert device_norm(B.linear(x, w)["y"], X @ W.t()) <= norm_bound(inner)
    b = B.linear_backward(gy, x, w)
    assert device_norm(b["gx"], G @ W) <= norm_bound(outer)
    assert device_norm(b["gw"], G.t() @ X) <= norm_bound(rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", [(3, 1, 5), (20, 64, 40), (300, 33, 70), (2051, 2049, 2050)])
def test_sums_of_one_sign(rows, inner, outer):
    """Values whose products lose most, all of one sign: 2^-21 of the sum, and a rounding of it for each instruction."""
    from equivariant_edge_convolution_amd import binding as B

    v = 1 + 2.0 ** -7 - 2.0 ** -23
    y = B.linear(torch.full((rows, inner), v, device="cuda"), torch.full((outer, inner), v, device="cuda"))["y"].double()
    ref = inner * v * v
    assert float((y - ref).abs().max()) <= (LEFT_OUT + (6 * (inner // 32 + 2) + 1) * EPS) * ref
