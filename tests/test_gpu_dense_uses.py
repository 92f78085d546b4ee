"""The dense operators as a program uses them: the atom head of
examples/atom_head.py (training and 8-bit evaluation behind the message), and a
training step captured in a HIP graph."""
import os
import sys

import numpy as np
import pytest
import torch

from equivariant_edge_convolution_amd import binding as B

from gpu_util import DEV, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import atom_head

pytestmark = pytest.mark.gpu


def test_atom_head_learns_and_evaluates_in_8_bits():
    losses, off = atom_head.run("D512", hidden=128, steps=150)
    say(f"[atom head] {losses[0]:.3g} -> {losses[-1]:.3g}, 8-bit deviation {off:.3g}")
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.2 * losses[0]
    # rows of e4m3 carry 2^-4 relative per value at most; the head's energies are of order one
    assert off < 0.5


def test_training_step_in_a_graph():
    """Captured once, replayed with other inputs and eager work in between: every replay equals the eager call."""
    g = torch.Generator().manual_seed(1)
    head = atom_head.Head(64, 128, DEV)
    x, ge = torch.randn(300, 64, generator=g).to(DEV), torch.randn(300, 1, generator=g).to(DEV)

    def step():
        e, kept = head.forward(x, train=True)
        grads, gx = head.backward(ge, kept)
        return [e, gx] + list(grads.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (2, 3, 4):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(300, 64, generator=g).to(DEV))
        ge.copy_(torch.randn(300, 1, generator=g).to(DEV))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
