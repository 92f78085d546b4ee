"""Host-side refusals of the orthogonalised update (CPU only): rejected before anything is launched, with the status and a message."""
import ctypes

import pytest

from equivariant_edge_convolution_amd import binding as B
from test_abi_dense import BF16, E4M3, F32, P

QUINTIC = (3.4445, -4.7750, 2.0315)


def ortho(batch=2, rows=64, cols=48, dtype=F32, g=P(1), ldg=48, stride=64 * 48, steps=5, coef=QUINTIC * 5, eps=1e-7, y=P(2), ws=P(3),
          size=1 << 40):
    c = None if coef is None else (ctypes.c_double * len(coef))(*coef)
    return B.STATUS[B.lib().eec_orthogonalize(None, batch, rows, cols, dtype, g, ldg, stride, steps, c, eps, y, ws, size)]


@pytest.mark.parametrize("call,status", [
    (lambda: ortho(dtype=E4M3), "EEC_ERR_SHAPE"), (lambda: ortho(dtype=4), "EEC_ERR_SHAPE"),
    (lambda: ortho(batch=-1), "EEC_ERR_SHAPE"), (lambda: ortho(batch=65536), "EEC_ERR_SHAPE"),
    (lambda: ortho(rows=-1), "EEC_ERR_SHAPE"), (lambda: ortho(cols=-1), "EEC_ERR_SHAPE"),
    (lambda: ortho(rows=(1 << 20) + 1, cols=1), "EEC_ERR_SHAPE"), (lambda: ortho(rows=1, cols=(1 << 20) + 1), "EEC_ERR_SHAPE"),
    (lambda: ortho(rows=(1 << 15) + 1, cols=(1 << 15) + 1), "EEC_ERR_SHAPE"),
    (lambda: ortho(steps=0), "EEC_ERR_SHAPE"), (lambda: ortho(steps=65, coef=QUINTIC * 65), "EEC_ERR_SHAPE"),
    (lambda: ortho(coef=None), "EEC_ERR_NULL"),
    (lambda: ortho(coef=(float("nan"), 0.0, 0.0) * 5), "EEC_ERR_SHAPE"), (lambda: ortho(coef=(1.0, float("inf"), 0.0) * 5), "EEC_ERR_SHAPE"),
    (lambda: ortho(coef=(4.0, 0.0, 0.0) * 5), "EEC_ERR_SHAPE"),               # 4 at once
    (lambda: ortho(coef=(1.5, 0.0, 0.0) * 5), "EEC_ERR_SHAPE"),               # 1.5^4 > 3.5
    (lambda: ortho(coef=(30.0, -60.0, 30.0) * 5), "EEC_ERR_SHAPE"),           # between 0 and 1, both of whose ends it takes to 0
    (lambda: ortho(coef=(16.0, -31.0, 15.0) * 5), "EEC_ERR_SHAPE"),           # b + c = -16
    (lambda: ortho(eps=0.0), "EEC_ERR_SHAPE"), (lambda: ortho(eps=-1.0), "EEC_ERR_SHAPE"), (lambda: ortho(eps=float("nan")), "EEC_ERR_SHAPE"),
    (lambda: ortho(eps=float("inf")), "EEC_ERR_SHAPE"),
    (lambda: ortho(g=None), "EEC_ERR_NULL"), (lambda: ortho(y=None), "EEC_ERR_NULL"),
    (lambda: ortho(ldg=47), "EEC_ERR_SHAPE"), (lambda: ortho(stride=-64 * 48), "EEC_ERR_SHAPE"),
    (lambda: ortho(stride=(1 << 40) + 1), "EEC_ERR_SHAPE"),
    (lambda: ortho(g=ctypes.c_void_p((1 << 32) + 2)), "EEC_ERR_SHAPE"),
    (lambda: ortho(rows=640, cols=480, ldg=480, stride=640 * 480, ws=None), "EEC_ERR_WORKSPACE"),
    (lambda: ortho(rows=640, cols=480, ldg=480, stride=640 * 480, size=1024), "EEC_ERR_WORKSPACE"),
    (lambda: ortho(rows=640, cols=480, ldg=480, stride=640 * 480, ws=ctypes.c_void_p((3 << 32) + 64)), "EEC_ERR_WORKSPACE"),
    (lambda: ortho(ws=None, size=0, y=P(1)), "EEC_ERR_ALIAS"),  # small updates need none
    (lambda: ortho(y=P(1)), "EEC_ERR_ALIAS"), (lambda: ortho(y=P(3)), "EEC_ERR_ALIAS"), (lambda: ortho(ws=P(1)), "EEC_ERR_ALIAS"),
    # y over the second matrix of the batch
    (lambda: ortho(stride=1 << 20, y=ctypes.c_void_p((1 << 32) + (4 << 20))), "EEC_ERR_ALIAS"),
    # sets of coefficients in use pass that check
    (lambda: ortho(y=P(1), coef=(1.875, -1.25, 0.375) * 5), "EEC_ERR_ALIAS"),
    (lambda: ortho(y=P(1), steps=2, coef=(8.28, -23.6, 17.3, 4.1, -2.95, 0.55)), "EEC_ERR_ALIAS"),
    # 1 goes to 1.98 and to 1.97, 0.376 to 1.99 and 2.08, which these take to 7
    (lambda: ortho(y=P(1), steps=3, coef=(8.28, -23.6, 17.3, 4.1, -2.95, 0.55, 1.875, -1.25, 0.375)), "EEC_ERR_SHAPE"),
    (lambda: ortho(y=P(1), steps=1, coef=(3.5, 0.0, 0.0)), "EEC_ERR_ALIAS"),
    (lambda: ortho(batch=1, stride=0, y=P(1)), "EEC_ERR_ALIAS"), (lambda: ortho(stride=48, ldg=96, y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: ortho(stride=0, y=P(1)), "EEC_ERR_ALIAS"),
    # y in the rows of the last of two interleaved matrices
    (lambda: ortho(stride=48, ldg=96, y=ctypes.c_void_p((1 << 32) + 4 * (48 + 63 * 96 + 47))), "EEC_ERR_ALIAS"),
])
def test_refusals(call, status):
    assert call() == status
    assert B.lib().eec_last_error() != b""


def test_nothing_to_do_is_not_an_error():
    assert ortho(batch=0, g=None, y=None) == "EEC_OK"
    assert ortho(rows=0, g=None, y=None) == "EEC_OK"
    assert ortho(cols=0, g=None, y=None) == "EEC_OK"


def test_workspace_queries():
    f = B.lib().eec_orthogonalize_workspace_bytes
    assert f(1, 1 << 20, 1 << 16, F32) == 0 and f(1, 64, 64, E4M3) == 0
    # X twice in two planes of 16 bits, and A and B
    assert f(1, 8192, 2048, BF16) >= 8 * 8192 * 2048 + 2 * 2 * 2048 * 2048
    assert f(4, 256, 128, F32) >= 4 * (8 * 256 * 128 + 2 * 4 * 128 * 128)
    assert f(1, 100, 200, F32) % 256 == 0
