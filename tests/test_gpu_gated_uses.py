"""The gated layer, products of 8-bit integers and orthogonalised updates as a program uses them together: the head of
examples/gated_head.py, trained and evaluated behind the message, and its whole training step captured in a HIP graph."""
import os
import sys

import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B
from oracle import dense as D

from gpu_util import DEV, np_, say
from test_gpu_dense import f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_head

pytestmark = pytest.mark.gpu


def test_gated_head_runs():
    losses, off = gated_head.run("D64", hidden=96, blocks=2, steps=12)
    say(f"[gated head] {losses[0]:.3g} -> {losses[-1]:.3g}, deviation in 8 bits {off:.3g}")
    assert len(losses) == 12 and np.all(np.isfinite(losses)) and np.isfinite(off)


def in_float64(x, p, ge):
    """The head's output and the sum of it times ge, by the definitions."""
    s = x
    for b in range(p["up"].shape[0]):
        y = D.norm(s, p["gain"][b])["y"]
        s = s + D.linear(D.gated(y, p["up"][b], p["up_bias"][b], "silu")["y"], p["down"][b], p["down_bias"][b])["y"]
    e = D.linear(D.norm(s, p["gain"][-1])["y"], p["w"])["y"]
    return e, float((e * ge).sum())


def test_gradients_of_the_head():
    """Against differences of the float64 definitions, along each gradient and along a direction at random.

    float32 at widths up to 48 in 3 products a block: (2 48 + 32) EPS = 8e-6 for each, 7 products deep; differences with
    steps of 1e-5 are off by 1e-9 of the third derivative. 2e-4 of the gradient's size bounds both."""
    g = torch.Generator().manual_seed(4)
    head = gated_head.GatedHead(32, 24, 2, DEV, seed=3)
    for k in ("up_bias", "down_bias"):
        head.p[k].copy_(torch.randn(head.p[k].shape, generator=g) * 0.1)
    x, ge = torch.randn(50, 32, generator=g).to(DEV), torch.randn(50, 1, generator=g).to(DEV)
    e, kept = head.forward(x, train=True)
    grads, gx = head.backward(ge, kept)
    p, X, G = {k: f64(v) for k, v in head.p.items()}, f64(x), f64(ge)
    want, _ = in_float64(X, p, G)
    assert np.abs(f64(e) - want).max() <= 2e-5 * np.abs(want).max()
    assert torch.equal(head.forward(x)[0], e)  # what training keeps changes nothing
    r = np.random.default_rng(0)
    for k, v in dict(grads, x=gx).items():
        at = X if k == "x" else p[k]
        for d in (f64(v), r.normal(size=at.shape)):
            h = 1e-5 / max(np.abs(d).max(), 1e-30)
            moved = lambda t: in_float64(at + t * d, p, G)[1] if k == "x" else in_float64(X, dict(p, **{k: at + t * d}), G)[1]
            slope = (moved(h) - moved(-h)) / (2 * h)
            size = np.linalg.norm(f64(v)) * np.linalg.norm(d)
            assert abs(slope - (f64(v) * d).sum()) <= 2e-4 * size, k


def test_evaluation_in_8_bits_follows_the_definition():
    """Codes, scales and products of the 8-bit pass against the same pass in 64 bits with the codes that it made: sums of
    integers are exact, so what is left are float32's roundings around them."""
    g = torch.Generator().manual_seed(5)
    head = gated_head.GatedHead(64, 48, 2, DEV, seed=6)
    x = torch.randn(300, 64, generator=g).to(DEV)
    q = head.quantized()
    e = f64(head.forward_int8(x, q))
    p, s = {k: f64(v) for k, v in head.p.items()}, f64(x)
    code = lambda v: (lambda c, scale: c.astype(np.float64) * scale.astype(np.float64)[:, None])(*D.quantize_i8(v))
    for b in range(2):
        up, down = (f64(q[k][b][0]) * f64(q[k][b][1])[:, None] for k in ("up", "down"))
        y = code(D.norm(s, p["gain"][b])["y"])
        h = code(D.gated(y, up, p["up_bias"][b], "silu")["y"])
        s = s + D.linear(h, down, p["down_bias"][b])["y"]
    want = D.linear(D.norm(s, p["gain"][-1])["y"], p["w"])["y"]
    # a code may fall the other way where float32 is off by its last bits: 1/127 of a row's largest value in one place
    assert np.abs(e - want).max() <= 0.02 * np.abs(want).max() and np.abs(e - want).mean() <= 1e-3 * np.abs(want).mean()
    for k, w in (("up", head.p["up"]), ("down", head.p["down"])):
        for b in range(2):
            codes, scale = D.quantize_i8(np_(w[b]))
            assert np.array_equal(np_(q[k][b][0]), codes) and np.array_equal(np_(q[k][b][1]), scale)


def test_training_step_in_a_graph():
    """Forward, backward and update captured once and replayed with other inputs, eager work in between: every replay
    equals the eager step, bit for bit."""
    g = torch.Generator().manual_seed(1)
    head = gated_head.GatedHead(64, 96, 2, DEV)
    x, target = torch.randn(300, 64, generator=g).to(DEV), torch.randn(300, 1, generator=g).to(DEV)

    def step():
        e, kept = head.forward(x, train=True)
        grads, gx = head.backward((e - target) * (2.0 / 300), kept)
        up = B.orthogonalize(grads["up"].unflatten(1, (2, -1)).flatten(0, 1))
        down = B.orthogonalize(grads["down"])
        y = B.quantize_rows(kept[0][0][1]["y"])
        return [e, gx, up, down, y["y"], y["scale"]] + list(grads.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same step: neither reads the other's workspaces
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        graphs.append((graph, captured))
    for seed in (2, 3, 4):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(300, 64, generator=g).to(DEV))
        target.copy_(torch.randn(300, 1, generator=g).to(DEV))
        eager = step()
        torch.cuda.synchronize()
        for graph, captured in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, captured in graphs:
            for a, b in zip(captured, eager):
                assert torch.equal(a, b)


def test_on_two_streams_at_once():
    """Calls of every operator on two streams, each with inputs of its own, as one after the other."""
    g = torch.Generator().manual_seed(7)
    sets = [(torch.randn(700, 520, generator=g).to(DEV), torch.randn(600, 520, generator=g).to(DEV) * 0.05,
             torch.randn(700, 300, generator=g).to(DEV)) for _ in range(2)]

    def work(x, w, gy):
        f = B.gated_linear(x, w, None, "gelu", save_preact=True)
        b = B.gated_linear_backward(gy, x, w, f["preact"], "gelu", bias=True)
        qx, qw = B.quantize_rows(x), B.quantize_rows(w)
        i = B.gated_linear(qx["y"], qw["y"], None, "silu", qx["scale"], qw["scale"], torch.float32)
        j = B.linear(qx["y"], qw["y"], x_scale=qx["scale"], w_scale=qw["scale"])
        return [f["y"], b["gx"], b["gw"], b["gbias"], i["y"], j["y"], B.orthogonalize(b["gw"]), B.orthogonalize(w[:40])]

    alone = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for stream, s in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append(work(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("rows,outer", [(70000, 16384), ((1 << 30) + 5, 1)])
def test_gated_outputs_past_32_bits(rows, outer):
    """More than 2^31 columns of z: constants, so that every output is known, and one row that differs at the end."""
    x = torch.ones((rows, 1), dtype=torch.bfloat16, device=DEV)
    x[rows - 1] = 2.0
    w = torch.ones((2 * outer, 1), dtype=torch.bfloat16, device=DEV)
    w[outer:] = 3.0
    y = B.gated_linear(x, w, None, "relu")["y"]
    assert torch.all(y[-1] == 12.0) and float(y[:-1].amax()) == 3.0 and float(y[:-1].amin()) == 3.0


def test_batches_past_32_bits():
    """Matrices whose offsets pass 2^31 elements: the last of them is treated as the first."""
    one = torch.randn(64, 512, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    g = one.expand(65535, 64, 512).contiguous()
    y = B.orthogonalize(g, steps=2)
    assert torch.equal(y[0], y[-1]) and torch.equal(y[0], B.orthogonalize(one, steps=2)) and torch.equal(y[40000], y[0])
    del g, y
    one = torch.randn(256, 260, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(DEV)
    g = one.expand(33000, 256, 260).contiguous()
    y = B.orthogonalize(g, steps=1)
    assert torch.equal(y[0], y[-1]) and torch.equal(y[0], y[20000]) and bool(torch.isfinite(y[0].float()).all())
