"""The block of examples/train_shared_expert_block.py: its gradients against autograd in 64 bits through the same routing, its
captured steps against eager ones, and that it runs."""
import importlib.util
import math
import os

import pytest
import torch

from dropless_mixture_experts_top_gb300.synth import MoEShape

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()
    spec = importlib.util.spec_from_file_location("train_shared", os.path.join(ROOT, "examples", "train_shared_expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference_out(p, h, idx, shape):
    """The block's output in 64 bits, the chosen experts given."""
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * p["norm_w"]
    s = torch.sigmoid(torch.gather(y @ p["W_r"], 1, idx))
    w = 1.5 * s / s.sum(1, keepdim=True)
    out = h + torch.nn.functional.gelu(y @ p["W_1"] + p["b_1"], approximate="tanh") @ p["W_2"] + p["b_2"]
    for e in range(shape.E):
        tok, j = (idx == e).nonzero(as_tuple=True)
        a = y[tok]
        z = torch.nn.functional.silu(a @ p["W_gate"][e]) * (a @ p["W_up"][e]) @ p["W_down"][e]
        out = out.index_add(0, tok, w[tok, j][:, None] * z)
    return out


def data(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(shape.T, shape.H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)] + [
        torch.randn(shape.T, shape.H, generator=g, device="cuda")]


@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
def test_output_and_gradients_of_the_whole_block(ex, groups):
    """bf16 rounds the activations between the operators: 2^-8 / sqrt 3 of a value in the mean, about six in a row (norm, hidden
    rows, experts' outputs; gradients in and out), which is 2^-8 sqrt 2 where they add up independently: 6e-3; twice that is
    allowed, and for the router's and the norm's weights, whose gradients are differences of such terms, three times it."""
    shape, shared = MoEShape(T=300, H=128, I=64, E=8, k=2), 72
    block = ex.Block(shape, shared, groups=groups[0], top_groups=groups[1], seed=5)
    block.bias.copy_(0.1 * torch.randn(shape.E, device="cuda"))
    block.master["b_1"].normal_()
    block.master["b_2"].normal_()
    for n in ("b_1", "b_2"):
        block.w[n].copy_(block.master[n])
    x, r, d = data(shape, 7)
    out = block.forward(x, r)
    d_out = (d / 16).to(torch.bfloat16).float()
    got = block.backward(d_out)
    assert block.status() == {}
    p = {n: w.to(torch.bfloat16).double().requires_grad_() for n, w in block.master.items()}
    h = block.normed["sum"].double().requires_grad_()
    ref = reference_out(p, h, block.layer.routing["topk_idx"].long(), shape)
    tol = 2 * math.sqrt(2) * 2.0 ** -8
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) <= tol
    (ref * d_out.double()).sum().backward()
    for n, want in [("h", h.grad)] + [(n, p[n].grad) for n in p]:
        g = got[n]
        g = (g.view(torch.bfloat16) if g.dtype == torch.int16 else g).double()
        assert float((g - want).norm() / want.norm()) <= (3 if n in ("W_r", "norm_w") else 1) * tol, n


def test_captured_steps_are_the_eager_ones(ex):
    shape = MoEShape(T=512, H=128, I=64, E=8, k=2)
    eager, captured = (ex.Block(shape, 136, groups=2, top_groups=1, seed=4) for _ in range(2))
    x, r, target = data(shape, 1)
    lr = torch.full((1,), 3e-3, device="cuda")
    for b in (eager, captured):
        ex.train_step(b, x, r, target, lr)
    graph, loss = ex.capture(captured, x, r, target, lr)
    for i in range(3):
        for t, v in zip((x, r, target), data(shape, 10 + i)):
            t.copy_(v)
        lr.fill_(1e-3 * (3 - i))
        graph.replay()
        want = ex.train_step(eager, x, r, target, lr)
        assert torch.equal(loss, want)
        for n in eager.master:
            assert torch.equal(eager.master[n], captured.master[n]), n
            assert torch.equal(eager.w[n], captured.w[n]), n
            assert torch.equal(eager.w[n], eager.master[n].to(torch.bfloat16)), n
        assert torch.equal(eager.bias, captured.bias)
    assert eager.status() == {} and captured.status() == {}


def test_a_short_training_run(ex):
    losses = ex.train(steps=5, shape=MoEShape(T=512, H=128, I=64, E=8, k=2), shared=64, log=None)
    assert len(losses) == 5 and all(math.isfinite(v) for v in losses)
