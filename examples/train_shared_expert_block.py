"""Trains a mixture-of-experts block with a shared expert beside the routed ones, sigmoid routing with a bias for balance
instead of a balance loss, and AdamW with states in 8 bits:

  norm (residual sum, RMS norm) -> router projection -> gate -> routed experts
                                -> shared expert (dense, gelu, dense), added to the routed experts' output

  h = x + r,  y = norm(h),  routing = gate(y W_r, bias),  out = h + experts(y, routing) + gelu(y W_1 + b_1) W_2 + b_2
  loss = mean (out - target)^2 / 2

Master weights are fp32; the step also writes the bf16 copies that the products take.  A whole training step, its bias'
step among it, is captured into one CUDA graph and replayed: nothing in it waits for the host.

  python examples/train_shared_expert_block.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape

BF16, F32 = torch.bfloat16, torch.float32


class Block:
    """Parameters, plans and one training step of the block."""

    # by the type of their gradients: the step takes tensors of one type at once
    MATRICES = ("W_gate", "W_up", "W_down", "W_1", "W_2")  # bf16
    OTHERS = ("W_r", "norm_w", "b_1", "b_2")               # fp32

    def __init__(self, shape, shared, groups=1, top_groups=1, bias_rate=1e-2, seed=0, state="8bit", device="cuda"):
        self.shape, self.bias_rate = shape, bias_rate
        T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*s, scale):
            return torch.randn(*s, generator=g, device=device) * scale
        self.master = {"norm_w": torch.ones(H, device=device), "W_r": randn(H, E, scale=H ** -0.5),
                       "W_gate": randn(E, H, I, scale=H ** -0.5), "W_up": randn(E, H, I, scale=H ** -0.5),
                       "W_down": randn(E, I, H, scale=I ** -0.5), "W_1": randn(H, shared, scale=H ** -0.5),
                       "b_1": torch.zeros(shared, device=device), "W_2": randn(shared, H, scale=shared ** -0.5),
                       "b_2": torch.zeros(H, device=device)}
        self.w = {n: p.to(BF16) for n, p in self.master.items()}
        self.bits = {n: p.view(torch.int16) for n, p in self.w.items()}  # as the layer and the router take them
        self.bias = torch.zeros(E, device=device)
        # plans, workspaces and states, made once
        self.norm = moe.Norm(T, H, kind="rms", bias=False)
        self.router = moe.Router(shape)
        self.gate = moe.Gate(T, E, k, score="sigmoid", groups=groups, top_groups=top_groups, group_best=2, scale=1.5)
        self.layer = moe.MoELayer(shape)
        self.up = moe.Linear(T, H, shared, activation="gelu")
        self.down = moe.Linear(T, shared, H)
        self.opt, self.state = {}, {}
        for name, grad in (("MATRICES", "bf16"), ("OTHERS", "fp32")):
            tensors = [self.master[n] for n in getattr(self, name)]
            self.opt[name] = moe.AdamW([p.shape for p in tensors], grad=grad, state=state, beta2=0.95,
                                       weight_decay=[0.01 * (p.dim() > 1) for p in tensors])
            self.state[name] = self.opt[name].new_state()

    def forward(self, x, r):
        """out (fp32 [T,H]); keeps what backward needs.  x, r: bf16 [T,H]."""
        w, b = self.w, self.bits
        self.normed = self.norm.forward(x, w["norm_w"], residual=r)
        self.y = self.normed["y"]
        y = self.y.view(torch.int16)
        self.logits = self.router.forward(y, b["W_r"])
        self.gate.forward(self.logits, self.bias, out=self.layer.routing)
        routed = self.layer.forward(y, b["W_gate"], b["W_up"], b["W_down"])
        self.hidden = self.up.forward(self.y, w["W_1"], w["b_1"])
        both = self.down.forward(self.hidden["y"], w["W_2"], w["b_2"], residual=moe.bf16_view(routed))
        return self.normed["sum"].float() + both["y"].float()

    def backward(self, d_out):
        """Gradients of every parameter and of h, from the gradient of out (fp32 [T,H])."""
        w, b, d = self.w, self.bits, d_out.to(BF16)
        y, routing = self.y.view(torch.int16), self.layer.routing
        down = self.down.backward(d, self.hidden["y"], w["W_2"])
        up = self.up.backward(down["dx"], self.y, w["W_1"], self.hidden["z"])
        g = self.layer.backward(d.view(torch.int16), y, b["W_gate"], b["W_up"], b["W_down"])
        # the gate's gradient in the place of that of the layer's own routing
        self.gate.backward(self.logits, routing["topk_idx"], routing["topk_w"], g["d_topk_w"], d_logits=g["d_logits"])
        d_wr = self.router.backward(y, b["W_r"], g["d_logits"], g["dx"])  # adds its part to dx
        d_y = (moe.bf16_view(g["dx"]).float() + up["dx"].float()).to(BF16)
        n = self.norm.backward(d_y, self.normed["sum"], w["norm_w"], self.normed["stats"], d_sum=d)
        return {"h": n["dx"], "norm_w": n["dweight"], "W_r": d_wr, "W_gate": g["dW_gate"], "W_up": g["dW_up"],
                "W_down": g["dW_down"], "W_1": up["dW"], "b_1": up["dbias"], "W_2": down["dW"], "b_2": down["dbias"]}

    def step(self, grads, lr):
        """AdamW of every parameter, and the gate's bias towards even loads.  lr: a number or a device number."""
        for name, opt in self.opt.items():
            names = getattr(self, name)
            opt.step([self.master[n] for n in names], [grads[n] for n in names], self.state[name], lr,
                     copies=[self.w[n] for n in names])
        self.gate.update_bias(self.bias, self.layer.routing["counts"], self.bias_rate)

    def status(self):
        layer = self.layer.status()
        del layer["route"]  # (the gate routes)
        found = {"layer": layer, "router": self.router.status(), "gate": self.gate.status(),
                 "up": self.up.status(), "down": self.down.status()}
        found.update({"step " + n: o.status(self.state[n]) for n, o in self.opt.items()})
        return {k: v for k, v in found.items() if any(v.values())}


def train_step(block, x, r, target, lr):
    err = block.forward(x, r) - target
    block.step(block.backward(err / err.numel()), lr)
    return err.square().mean() / 2


def capture(block, x, r, target, lr):
    """(graph, loss): one training step on what x, r, target and lr hold when it is replayed.  A step has run before: the first
    call of a kernel sets it up, which a capture cannot."""
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        loss = train_step(block, x, r, target, lr)
    return graph, loss


def train(steps=100, shape=MoEShape(T=2048, H=256, I=128, E=16, k=2), shared=256, lr=3e-3, log=print):
    """Returns the losses of every step."""
    teacher = Block(shape, shared, seed=1)
    block = Block(shape, shared, groups=4, top_groups=2, seed=2)
    x, r = (torch.zeros(shape.T, shape.H, dtype=BF16, device="cuda") for _ in range(2))
    target, rate = torch.zeros(shape.T, shape.H, device="cuda"), torch.zeros(1, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    losses, graph = [], None
    for i in range(steps):
        for t in (x, r):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        target.copy_(teacher.forward(x, r))
        rate.fill_(lr * (1 - i / steps))
        if i == 0:
            losses.append(train_step(block, x, r, target, rate))
        else:
            if graph is None:
                graph, loss = capture(block, x, r, target, rate)
            graph.replay()
            losses.append(loss.clone())
        if log and (i % 20 == 0 or i + 1 == steps):
            log(f"step {i:3d}  loss {float(losses[-1]):.4f}  fullest expert {int(block.layer.routing['counts'].max())} of "
                f"{shape.T * shape.k // shape.E} slots evenly")
    bad = block.status()
    if bad:
        raise RuntimeError(f"device status: {bad}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100)
