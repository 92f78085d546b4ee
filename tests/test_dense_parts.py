"""float32 products in bf16 parts: six of the nine part products, at float32's accuracy.

The operands' three parts are truncated, so what the three products left out are worth has the sign of the whole: with
|m| < 2^-7 and |l| < 2^-15 of a value's power of two at most 2 2^-22 + 2^-30 of each product.
"""
import numpy as np
import pytest
import torch

EPS = 2.0 ** -24
LEFT_OUT = 2.0 ** -21 + 2.0 ** -30
TAKEN = ((2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0))  # parts h, m, l of one operand and of the other


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


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", [(3, 1, 5), (20, 64, 40), (300, 33, 70), (2051, 2049, 2050)])
def test_sums_of_one_sign(rows, inner, outer):
    """Values whose products lose most, all of one sign: 2^-21 of the sum, and a rounding of it for each instruction."""
    from equivariant_edge_convolution_amd import binding as B

    v = 1 + 2.0 ** -7 - 2.0 ** -23
    y = B.linear(torch.full((rows, inner), v, device="cuda"), torch.full((outer, inner), v, device="cuda"))["y"].double()
    ref = inner * v * v
    assert float((y - ref).abs().max()) <= (LEFT_OUT + (6 * (inner // 32 + 2) + 1) * EPS) * ref
