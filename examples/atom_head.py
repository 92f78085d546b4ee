#!/usr/bin/env python3
"""A network on the atoms behind the message: per-atom energies from the l = 0
channels of A, trained with the dense operators and evaluated in 8 bits.

    x   = A[:, 0, :]                       (a view: row stride 16 C)
    y1  = norm(x),        d1 = silu(y1 W1 + b1) W2 + b2
    s   = x + d1,   y2  = norm(s)          (one call)
    o   = silu(y2 W3 + b3) W4 + b4 + s,    E_i = o . w

The head gives energies.  Its backward ends at the gradient of x: the library takes no
gradient of A on to the positions, so there are no forces through the head.

The target is the model's own quadratic readout, standardised over the cell, so
the data need nothing but a seeded cell.  Every product, norm and gradient is one
of the library's calls; torch allocates, and takes the optimiser's elementwise step.

    python examples/atom_head.py [--config D512] [--steps 300] [--lr 3e-3]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import eec_inputs as I
from equivariant_edge_convolution_amd import binding as B


class Head:
    """The network's weights and its forward and backward passes."""

    def __init__(self, channels: int, hidden: int, device, dtype=torch.float32, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(device=device, dtype=dtype)
        c, h = channels, hidden
        self.p = dict(g1=torch.ones(c, device=device, dtype=dtype), w1=new(h, c, scale=c ** -0.5),
                      b1=torch.zeros(h, device=device, dtype=dtype), w2=new(c, h, scale=h ** -0.5),
                      b2=torch.zeros(c, device=device, dtype=dtype), g2=torch.ones(c, device=device, dtype=dtype),
                      w3=new(h, c, scale=c ** -0.5), b3=torch.zeros(h, device=device, dtype=dtype),
                      w4=new(c, h, scale=h ** -0.5), b4=torch.zeros(c, device=device, dtype=dtype),
                      w=new(1, c, scale=c ** -0.5))

    def forward(self, x: torch.Tensor, train: bool = False):
        p = self.p
        n1 = B.add_rms_norm(x, p["g1"], save_rstd=train)
        h1 = B.linear(n1["y"], p["w1"], p["b1"], "silu", save_preact=train)
        d1 = B.linear(h1["y"], p["w2"], p["b2"])
        n2 = B.add_rms_norm(d1["y"], p["g2"], residual=x, save_rstd=train)
        h2 = B.linear(n2["y"], p["w3"], p["b3"], "silu", save_preact=train)
        o = B.linear(h2["y"], p["w4"], p["b4"], residual=n2["sum"])
        e = B.linear(o["y"], p["w"])["y"]
        return e, (x, n1, h1, n2, h2, o)

    def backward(self, ge: torch.Tensor, kept) -> tuple[dict, torch.Tensor]:
        """Gradients of the weights, and of x."""
        p = self.p
        x, n1, h1, n2, h2, o = kept
        be = B.linear_backward(ge, o["y"], p["w"], bias=False)
        b4 = B.linear_backward(be["gx"], h2["y"], p["w4"])
        b3 = B.linear_backward(b4["gx"], n2["y"], p["w3"], h2["preact"], "silu")
        m2 = B.add_rms_norm_backward(b3["gx"], n2["sum"], p["g2"], n2["rstd"], gsum=be["gx"])
        b2 = B.linear_backward(m2["gx"], h1["y"], p["w2"])
        b1 = B.linear_backward(b2["gx"], n1["y"], p["w1"], h1["preact"], "silu")
        m1 = B.add_rms_norm_backward(b1["gx"], x, p["g1"], n1["rstd"], gsum=m2["gx"])
        grads = dict(g1=m1["gweight"], w1=b1["gw"], b1=b1["gbias"], w2=b2["gw"], b2=b2["gbias"], g2=m2["gweight"],
                     w3=b3["gw"], b3=b3["gbias"], w4=b4["gw"], b4=b4["gbias"], w=be["gw"])
        return grads, m1["gx"]

    def forward_8bit(self, x: torch.Tensor):
        """The same network with 8-bit rows into the wide layers (weights quantised once, here)."""
        p = self.p
        q = {}
        for k in ("w1", "w3"):
            scale = p[k].abs().amax(dim=1).clamp_min(2.0 ** -100) / 448.0
            q[k] = ((p[k] / scale[:, None]).to(torch.float8_e4m3fn), scale)
        t = x.dtype
        n1 = B.add_rms_norm(x, p["g1"], quantize=True)
        h1 = B.linear(n1["y"], q["w1"][0], p["b1"], "silu", x_scale=n1["scale"], w_scale=q["w1"][1], out_dtype=t)
        d1 = B.linear(h1["y"], p["w2"], p["b2"])
        n2 = B.add_rms_norm(d1["y"], p["g2"], residual=x, quantize=True)
        h2 = B.linear(n2["y"], q["w3"][0], p["b3"], "silu", x_scale=n2["scale"], w_scale=q["w3"][1], out_dtype=t)
        o = B.linear(h2["y"], p["w4"], p["b4"], residual=n2["sum"])
        return B.linear(o["y"], p["w"])["y"]


def run(config: str = "D512", hidden: int = 256, steps: int = 300, lr: float = 3e-3, device="cuda"):
    """Trains the head; returns the losses and the largest 8-bit deviation of a standardised energy."""
    cfg = I.make_config(config)
    pos, species = torch.as_tensor(cfg.pos).to(device), torch.as_tensor(cfg.species).to(device)
    model = B.Model.from_arrays(cfg.model, device)
    graph = B.build_neighbors(pos, cfg.box, cfg.model.cutoff, species, cfg.model.n_species)
    A = B.edge_message(graph, pos, cfg.box, species, model)
    target = B.energy_forces(graph, pos, cfg.box, species, model)["atom_energy"]
    target = ((target - target.mean()) / target.std())[:, None].contiguous()
    x = A[:, 0, :]
    head = Head(model.channels, hidden, x.device)
    moment = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in head.p.items()}
    losses = []
    for step in range(1, steps + 1):
        e, kept = head.forward(x, train=True)
        d = e - target
        losses.append((d * d).mean())
        grads, _ = head.backward(d * (2.0 / d.numel()), kept)
        for k, g in grads.items():  # Adam
            m, v = moment[k]
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.01)
            head.p[k].sub_(lr * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8))
    full, eight = head.forward(x)[0], head.forward_8bit(x)
    return [float(v) for v in losses], float((full - eight).abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="D512", choices=sorted(I.CONFIGS))
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args()
    losses, off = run(a.config, a.hidden, a.steps, a.lr)
    for k in sorted({0, len(losses) // 4, len(losses) // 2, len(losses) - 1}):
        print(f"step {k + 1}: mean squared error {losses[k]:.4g} (standardised energies)")
    print(f"8-bit evaluation: largest deviation {off:.3g}")


if __name__ == "__main__":
    main()
