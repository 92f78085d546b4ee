#!/usr/bin/env python3
"""A network of gated blocks on the atoms behind the message: per-atom energies from the l = 0 channels of A,
trained with orthogonalised updates and evaluated in 8-bit integers.

    s_0 = A[:, 0, :]                                    (a view: row stride 16 C)
    s_b = s_(b-1) + (silu(y Wg^T + bg) * (y Wv^T + bv)) Wd^T + bd,   y = norm(s_(b-1)),    b = 1 .. blocks
    E_i = norm(s_blocks) . w

The head gives energies; its backward ends at the gradient of s_0 (the library takes no gradient of A on to the
positions). The target is the model's own quadratic readout, standardised over the cell, so the data need nothing but a
seeded cell. Every product, norm, gradient and orthogonalisation is one of the library's calls; torch allocates, and takes
the elementwise steps of the optimiser: momentum for the matrices, Adam for the vectors.

    python examples/gated_head.py [--config D512] [--blocks 2] [--hidden 128] [--steps 200] [--lr 0.02]
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


class GatedHead:
    """The network's weights, all blocks of a kind in one tensor, and its forward and backward passes."""

    MATRICES = ("up", "down")  # up: the gate's rows, then the value's

    def __init__(self, channels: int, hidden: int, blocks: int, device, dtype=torch.float32, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(device=device, dtype=dtype)
        zeros = lambda *s: torch.zeros(*s, device=device, dtype=dtype)
        c, h, b = channels, hidden, blocks
        self.blocks, self.hidden = blocks, hidden
        self.p = dict(up=new(b, 2 * h, c, scale=c ** -0.5), up_bias=zeros(b, 2 * h), down=new(b, c, h, scale=h ** -0.5),
                      down_bias=zeros(b, c), gain=torch.ones(b + 1, c, device=device, dtype=dtype),
                      w=new(1, c, scale=c ** -0.5))

    def forward(self, x: torch.Tensor, train: bool = False):
        p, kept, s, d = self.p, [], x, None
        for b in range(self.blocks):
            n = B.add_rms_norm(s if d is None else d, p["gain"][b], residual=None if d is None else s, save_rstd=train)
            s = n["sum"]
            h = B.gated_linear(n["y"], p["up"][b], p["up_bias"][b], "silu", save_preact=train)
            d = B.linear(h["y"], p["down"][b], p["down_bias"][b])["y"]
            kept.append((s, n, h))
        n = B.add_rms_norm(d, p["gain"][-1], residual=s, save_rstd=train)
        return B.linear(n["y"], p["w"])["y"], (kept, n)

    def backward(self, ge: torch.Tensor, kept) -> tuple[dict, torch.Tensor]:
        """Gradients of the weights, and of x."""
        p, (blocks, n) = self.p, kept
        out = {k: torch.empty_like(v) for k, v in p.items()}
        e = B.linear_backward(ge, n["y"], p["w"], bias=False)
        out["w"] = e["gw"]
        m = B.add_rms_norm_backward(e["gx"], n["sum"], p["gain"][-1], n["rstd"])
        out["gain"][-1] = m["gweight"]
        gs = m["gx"]  # of the residual stream, and of what the last block added to it
        for b in reversed(range(self.blocks)):
            s, n, h = blocks[b]
            d = B.linear_backward(gs, h["y"], p["down"][b])
            u = B.gated_linear_backward(d["gx"], n["y"], p["up"][b], h["preact"], "silu")
            m = B.add_rms_norm_backward(u["gx"], s, p["gain"][b], n["rstd"], gsum=gs)
            gs = m["gx"]
            for k, v in (("down", d["gw"]), ("down_bias", d["gbias"]), ("up", u["gw"]), ("up_bias", u["gbias"]), ("gain", m["gweight"])):
                out[k][b] = v
        return out, gs

    def quantized(self) -> dict:
        """The blocks' matrices in 8-bit integers, a scale per output channel."""
        rows = lambda v: B.quantize_rows(v.flatten(0, 1))
        up, down, b = rows(self.p["up"]), rows(self.p["down"]), self.blocks
        split = lambda q: list(zip(q["y"].unflatten(0, (b, -1)), q["scale"].unflatten(0, (b, -1))))
        return dict(up=split(up), down=split(down))

    def forward_int8(self, x: torch.Tensor, q: dict) -> torch.Tensor:
        """The same network, its blocks' products in 8-bit integers; rows are quantised on the way."""
        p, s, d, t = self.p, x, None, x.dtype
        for b in range(self.blocks):
            n = B.add_rms_norm(s if d is None else d, p["gain"][b], residual=None if d is None else s)
            s = n["sum"]
            y = B.quantize_rows(n["y"])
            h = B.gated_linear(y["y"], q["up"][b][0], p["up_bias"][b], "silu", y["scale"], q["up"][b][1], t)
            h = B.quantize_rows(h["y"])
            d = B.linear(h["y"], q["down"][b][0], p["down_bias"][b], x_scale=h["scale"], w_scale=q["down"][b][1], out_dtype=t)["y"]
        n = B.add_rms_norm(d, p["gain"][-1], residual=s)
        return B.linear(n["y"], p["w"])["y"]


class Optimizer:
    """Momentum and an orthogonalised step for the matrices, Adam for the rest."""

    def __init__(self, head: GatedHead, lr: float):
        self.head, self.lr, self.t = head, lr, 0
        self.state = {k: [torch.zeros_like(v) for _ in range(1 if k in head.MATRICES else 2)] for k, v in head.p.items()}

    def step(self, grads: dict):
        self.t += 1
        for k, g in grads.items():
            p, state = self.head.p[k], self.state[k]
            if k in self.head.MATRICES:
                state[0].mul_(0.9).add_(g)
                # gate and value are maps of their own: two matrices of a block, all blocks in one call
                u = torch.add(g, state[0], alpha=0.9)
                shape = u.shape
                if k == "up":
                    u = u.unflatten(1, (2, -1)).flatten(0, 1)
                u = B.orthogonalize(u).view(shape)
                p.sub_(u, alpha=self.lr * max(1.0, self.head.hidden / p.shape[-1] if k == "up" else p.shape[-2] / p.shape[-1]) ** 0.5)
            else:
                m, v = state
                m.lerp_(g, 0.1)
                v.lerp_(g * g, 0.01)
                p.sub_(0.1 * self.lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8))


def run(config: str = "D512", hidden: int = 128, blocks: int = 2, steps: int = 200, lr: float = 0.02, device="cuda"):
    """Trains the head; returns the losses and the largest deviation of a standardised energy in 8-bit integers."""
    cfg = I.make_config(config)
    pos, species = torch.as_tensor(cfg.pos).to(device), torch.as_tensor(cfg.species).to(device)
    model = B.Model.from_arrays(cfg.model, device)
    graph = B.build_neighbors(pos, cfg.box, cfg.model.cutoff, species, cfg.model.n_species)
    A = B.edge_message(graph, pos, cfg.box, species, model)
    target = B.energy_forces(graph, pos, cfg.box, species, model)["atom_energy"]
    target = ((target - target.mean()) / target.std())[:, None].contiguous()
    x = A[:, 0, :]
    head = GatedHead(model.channels, hidden, blocks, x.device)
    optimizer = Optimizer(head, lr)
    losses = []
    for _ in range(steps):
        e, kept = head.forward(x, train=True)
        d = e - target
        losses.append((d * d).mean())
        optimizer.step(head.backward(d * (2.0 / d.numel()), kept)[0])
    full, eight = head.forward(x)[0], head.forward_int8(x, head.quantized())
    return [float(v) for v in losses], float((full - eight).abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--config", default="D512", choices=sorted(I.CONFIGS))
    ap.add_argument("--hidden", type=int, default=128)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    losses, off = run(a.config, a.hidden, a.blocks, a.steps, a.lr)
    for k in sorted({0, len(losses) // 4, len(losses) // 2, len(losses) - 1}):
        print(f"step {k + 1}: mean squared error {losses[k]:.4g} (standardised energies)")
    print(f"8-bit integers: largest deviation {off:.3g}")


if __name__ == "__main__":
    main()
