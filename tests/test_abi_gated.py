"""Host-side refusals of the gated layer, of rows in 8 bits and of 8-bit integer operands (CPU only): every case is
rejected before anything is launched, with the status and a message."""
import ctypes

import pytest

from equivariant_edge_convolution_amd import binding as B
from test_abi_dense import BF16, E4M3, F16, F32, P, linear, norm

I8 = 4


def gated(rows=64, outer=48, inner=32, dtype=F32, out=F32, x=P(1), ldx=32, xs=None, w=P(2), ldw=32, ws_=None, bias=None,
          act=2, y=P(3), pre=None, ws=P(4), size=1 << 30):
    return B.STATUS[B.lib().eec_gated_linear(None, rows, outer, inner, dtype, out, x, ldx, xs, w, ldw, ws_, bias, act, y,
                                             pre, ws, size)]


def gated_bwd(rows=64, outer=48, inner=32, dtype=F32, act=2, gy=P(1), ldgy=48, x=P(2), ldx=32, w=P(3), ldw=32, pre=P(8),
              gx=P(4), gw=P(5), gb=P(6), ws=P(7), size=1 << 30):
    return B.STATUS[B.lib().eec_gated_linear_backward(None, rows, outer, inner, dtype, act, gy, ldgy, x, ldx, w, ldw, pre,
                                                      gx, gw, gb, ws, size)]


def quantize(rows=4, width=8, dtype=F32, codes=I8, x=P(1), ldx=8, y=P(2), scale=P(3)):
    return B.STATUS[B.lib().eec_quantize_rows(None, rows, width, dtype, codes, x, ldx, y, scale)]


@pytest.mark.parametrize("call,status", [
    (lambda: gated(dtype=9), "EEC_ERR_SHAPE"), (lambda: gated(out=F16), "EEC_ERR_SHAPE"),
    (lambda: gated(act=4), "EEC_ERR_SHAPE"), (lambda: gated(act=-1), "EEC_ERR_SHAPE"),
    (lambda: gated(inner=-1), "EEC_ERR_SHAPE"), (lambda: gated(outer=(1 << 26) + 1), "EEC_ERR_SHAPE"),
    (lambda: gated(rows=1 << 20, outer=(1 << 15) + 1, inner=1, ldx=1, ldw=1), "EEC_ERR_SHAPE"),  # 2^36 columns of z and more
    (lambda: gated(rows=1 << 31), "EEC_ERR_SHAPE"),
    (lambda: gated(x=None), "EEC_ERR_NULL"), (lambda: gated(w=None), "EEC_ERR_NULL"), (lambda: gated(y=None), "EEC_ERR_NULL"),
    (lambda: gated(ldw=31), "EEC_ERR_SHAPE"), (lambda: gated(ldx=31), "EEC_ERR_SHAPE"),
    (lambda: gated(x=ctypes.c_void_p((1 << 32) + 2)), "EEC_ERR_SHAPE"),
    (lambda: gated(xs=P(5)), "EEC_ERR_SHAPE"), (lambda: gated(dtype=E4M3, out=BF16), "EEC_ERR_NULL"),
    (lambda: gated(dtype=I8, out=BF16), "EEC_ERR_NULL"), (lambda: gated(dtype=I8, out=I8, xs=P(5), ws_=P(6)), "EEC_ERR_SHAPE"),
    (lambda: gated(dtype=I8, out=BF16, inner=1 << 17, ldx=1 << 17, ldw=1 << 17, xs=P(5), ws_=P(6)), "EEC_ERR_SHAPE"),
    (lambda: gated(rows=2048, outer=1024, inner=2048, ldx=2048, ldw=2048, ws=None, size=0), "EEC_ERR_WORKSPACE"),
    (lambda: gated(ws=ctypes.c_void_p((4 << 32) + 64), rows=2048, outer=1024, inner=2048, ldx=2048, ldw=2048), "EEC_ERR_WORKSPACE"),
    (lambda: gated(y=P(2)), "EEC_ERR_ALIAS"), (lambda: gated(pre=P(3)), "EEC_ERR_ALIAS"), (lambda: gated(bias=P(3)), "EEC_ERR_ALIAS"),
    # y over the value's rows of w, half of w past the gate's
    (lambda: gated(y=ctypes.c_void_p((2 << 32) + 48 * 32 * 4)), "EEC_ERR_ALIAS"),
    # the second half of preact over y
    (lambda: gated(pre=ctypes.c_void_p((3 << 32) - 64 * 48 * 4)), "EEC_ERR_ALIAS"),
    (lambda: gated_bwd(dtype=E4M3), "EEC_ERR_SHAPE"), (lambda: gated_bwd(dtype=I8), "EEC_ERR_SHAPE"),
    (lambda: gated_bwd(pre=None), "EEC_ERR_NULL"), (lambda: gated_bwd(act=0, pre=None), "EEC_ERR_NULL"),
    (lambda: gated_bwd(gy=None), "EEC_ERR_NULL"), (lambda: gated_bwd(x=None), "EEC_ERR_NULL"), (lambda: gated_bwd(w=None), "EEC_ERR_NULL"),
    (lambda: gated_bwd(ldgy=47), "EEC_ERR_SHAPE"), (lambda: gated_bwd(ws=None), "EEC_ERR_WORKSPACE"),
    (lambda: gated_bwd(size=0), "EEC_ERR_WORKSPACE"), (lambda: gated_bwd(gx=P(1)), "EEC_ERR_ALIAS"),
    (lambda: gated_bwd(gw=P(4)), "EEC_ERR_ALIAS"), (lambda: gated_bwd(gb=P(7)), "EEC_ERR_ALIAS"),
    (lambda: gated_bwd(gx=P(8)), "EEC_ERR_ALIAS"),
    (lambda: gated_bwd(rows=8, outer=1 << 19, inner=(1 << 16) + 1, ldgy=1 << 19, ldx=1 << 17, ldw=1 << 17), "EEC_ERR_SHAPE"),
    (lambda: quantize(dtype=I8), "EEC_ERR_SHAPE"), (lambda: quantize(codes=F32), "EEC_ERR_SHAPE"), (lambda: quantize(codes=7), "EEC_ERR_SHAPE"),
    (lambda: quantize(width=0), "EEC_ERR_SHAPE"), (lambda: quantize(rows=-1), "EEC_ERR_SHAPE"), (lambda: quantize(ldx=7), "EEC_ERR_SHAPE"),
    (lambda: quantize(x=None), "EEC_ERR_NULL"), (lambda: quantize(y=None), "EEC_ERR_NULL"), (lambda: quantize(scale=None), "EEC_ERR_NULL"),
    (lambda: quantize(y=P(1)), "EEC_ERR_ALIAS"), (lambda: quantize(scale=P(2)), "EEC_ERR_ALIAS"),
    (lambda: quantize(scale=ctypes.c_void_p((3 << 32) + 2)), "EEC_ERR_SHAPE"),
    (lambda: linear(dtype=I8, out=BF16), "EEC_ERR_NULL"), (lambda: linear(dtype=I8, out=I8, xs=P(5), ws_=P(6)), "EEC_ERR_SHAPE"),
    (lambda: linear(dtype=I8, out=F32, inner=1 << 17, ldx=1 << 17, ldw=1 << 17, xs=P(5), ws_=P(6)), "EEC_ERR_SHAPE"),
    # the longest sums that 32 bits hold pass that check
    (lambda: linear(dtype=I8, out=F32, inner=(1 << 17) - 1, ldx=1 << 17, ldw=1 << 17, xs=P(5), ws_=P(6), y=P(1)), "EEC_ERR_ALIAS"),
    (lambda: norm(dtype=I8), "EEC_ERR_SHAPE"),
])
def test_refusals(call, status):
    assert call() == status
    assert B.lib().eec_last_error() != b""


def test_nothing_to_do_is_not_an_error():
    assert gated(rows=0, x=None, y=None) == "EEC_OK"
    assert gated(outer=0, w=None, y=None) == "EEC_OK"
    assert gated_bwd(rows=0, outer=0, inner=0, gy=None, x=None, w=None, pre=None, gx=None, gw=None, gb=None) == "EEC_OK"
    assert quantize(rows=0, x=None, y=None, scale=None) == "EEC_OK"


def test_workspace_queries():
    L = B.lib()
    assert L.eec_gated_linear_workspace_bytes(8192, 4096, 4096, BF16, BF16) == 0  # aligned operands, enough tiles
    assert L.eec_gated_linear_workspace_bytes(1, 4096, 4096, F32, F32) == 0       # one row
    assert L.eec_gated_linear_workspace_bytes(4096, 1 << 27, 64, F32, F32) == 0   # refused
    assert L.eec_gated_linear_backward_workspace_bytes(64, 64, 64, I8) == 0
    # gz of both halves
    assert L.eec_gated_linear_backward_workspace_bytes(1000, 512, 256, BF16) >= 1000 * 1024 * 2
    assert (L.eec_gated_linear_backward_workspace_bytes(1000, 512, 256, BF16) ==
            L.eec_linear_backward_workspace_bytes(1000, 1024, 256, BF16, 2))
    assert L.eec_linear_workspace_bytes(8192, 4096, 4096, I8, BF16) == 0
