"""Trains one mixture-of-experts block on synthetic data, with every operator of the library in its place:

  norm (residual sum, layer norm) -> router projection -> routing -> balance and z loss -> experts -> combine,
  the backward of all of it, and orthogonalised updates of the expert and router weights.

  h = x + r,  y = norm(h),  logits = y W_r,  out = h + experts(y, route(logits))
  loss = mean (out - target)^2 / 2 + g_balance * balance + g_z * z

The block learns to follow a teacher of the same shape.  Its weights are kept in fp32 and handed to the library in
bf16; the bf16 tensors that the layer takes are int16 views of their bits.

  python examples/train_block.py [steps]
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape

BF16, F32 = torch.bfloat16, torch.float32


def bits(t):
    """A bf16 copy of t as the layer takes it."""
    return t.to(BF16).view(torch.int16)


class Block:
    """Parameters, plans and one training step of the block."""

    EXPERTS = ("W_gate", "W_up", "W_down")

    def __init__(self, shape, sequences=1, g_balance=0.01, g_z=1e-4, seed=0, device="cuda"):
        self.shape, self.g_balance, self.g_z = shape, g_balance, g_z
        T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*s, scale):
            return torch.randn(*s, generator=g, device=device) * scale
        self.master = {"norm_w": torch.ones(H, device=device), "norm_b": torch.zeros(H, device=device),
                       "W_r": randn(H, E, scale=H ** -0.5), "W_gate": randn(E, H, I, scale=H ** -0.5),
                       "W_up": randn(E, H, I, scale=H ** -0.5), "W_down": randn(E, I, H, scale=I ** -0.5)}
        # plans and workspaces, made once
        self.norm = moe.Norm(T, H, kind="layer", dtype="bf16")
        self.router = moe.Router(shape)
        self.layer = moe.MoELayer(shape)
        self.balance = moe.BalanceLoss(T, E, k, sequences=sequences)
        self.ortho = {"W_r": moe.Orthogonaliser(1, H, E, dtype="fp32"), "W_gate": moe.Orthogonaliser(E, H, I),
                      "W_up": moe.Orthogonaliser(E, H, I), "W_down": moe.Orthogonaliser(E, I, H)}
        self.momentum = {n: torch.zeros_like(w if w.dim() == 3 else w[None]) for n, w in self.master.items()
                         if n in self.ortho}
        self.cast()

    def cast(self):
        self.w = {n: bits(w) for n, w in self.master.items()}

    def forward(self, x, r, mask=None):
        """out (fp32 [T,H]); keeps what backward needs.  x, r: bf16 [T,H]."""
        w = self.w
        self.normed = self.norm.forward(x, w["norm_w"], w["norm_b"], residual=r)
        self.y = self.normed["y"].view(torch.int16)
        self.logits = self.router.forward(self.y, w["W_r"])
        self.layer.route(self.logits)
        self.aux = self.balance.forward(self.logits, self.layer.routing["topk_idx"], mask=mask)
        moe_out = self.layer.forward(self.y, *(w[n] for n in self.EXPERTS))
        return self.normed["sum"].float() + moe.bf16_view(moe_out).float()

    def backward(self, d_out):
        """Gradients of every parameter and of h, from the gradient of out (fp32 [T,H])."""
        w, d_h = self.w, d_out.to(BF16)
        g = self.layer.backward(d_h.view(torch.int16), self.y, *(w[n] for n in self.EXPERTS))
        aux = self.aux
        self.balance.backward(self.logits, aux["counts"], aux["tokens"], aux["lse"], self.g_balance, self.g_z,
                              d_logits=g["d_logits"])
        d_wr = self.router.backward(self.y, w["W_r"], g["d_logits"], g["dx"])  # adds its part to dx
        n = self.norm.backward(g["dx"], self.normed["sum"], w["norm_w"], self.normed["stats"], d_sum=d_h)
        return {"h": n["dx"], "norm_w": n["dweight"], "norm_b": n["dbias"], "W_r": d_wr,
                "W_gate": g["dW_gate"], "W_up": g["dW_up"], "W_down": g["dW_down"]}

    def step(self, grads, lr, beta=0.9):
        """Orthogonalised updates of the matrices, plain ones of the norm."""
        for n, w in self.master.items():
            if n in self.ortho:
                rows, cols = w.shape[-2:]
                upd = self.ortho[n].update(grads[n].view(self.momentum[n].shape), momentum=self.momentum[n], beta=beta,
                                           scale=math.sqrt(max(1.0, cols / rows)))
                w.sub_(lr * moe.bf16_view(upd).float().view(w.shape))
            else:
                w.sub_(lr * grads[n])
        self.cast()

    def status(self):
        found = {"layer": self.layer.status(), "router": self.router.status(), "balance": self.balance.status()}
        found.update({"update " + n: o.status() for n, o in self.ortho.items()})
        return {k: v for k, v in found.items() if any(v.values())}


def data(shape, teacher, seed, device="cuda"):
    """Inputs x and r of one batch and the teacher's outputs."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x, r = (torch.randn(shape.T, shape.H, generator=g, device=device).to(BF16) for _ in range(2))
    return x, r, teacher.forward(x, r)


def train(steps=60, shape=MoEShape(T=2048, H=256, I=128, E=16, k=2), lr=0.01, log=print):
    """Returns the losses (prediction, balance) of every step."""
    teacher = Block(shape, seed=1)
    block = Block(shape, sequences=4, seed=2)
    losses = []
    for i in range(steps):
        x, r, target = data(shape, teacher, 100 + i)
        out = block.forward(x, r)
        err = out - target
        losses.append((err.square().mean() / 2, block.aux["loss"][0].clone()))
        block.step(block.backward(err / err.numel()), lr * (1 - i / steps))
        if log and (i % 10 == 0 or i + 1 == steps):
            log(f"step {i:3d}  loss {float(losses[-1][0]):.4f}  balance {float(losses[-1][1]):.4f}  "
                f"fullest expert {int(block.aux['counts'].sum(0).max())} of {shape.T * shape.k // shape.E} slots evenly")
    bad = block.status()
    if bad:
        raise RuntimeError(f"device status: {bad}")
    return [(float(a), float(b)) for a, b in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
