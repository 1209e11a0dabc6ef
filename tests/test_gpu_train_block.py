"""The block of examples/train_block.py: its gradients against autograd in 64 bits through the same routing, and a short
training run."""
import importlib.util
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
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference_loss(p, h, d_out, idx, shape, sequences, g_balance, g_z):
    """<out, d_out> + the auxiliary losses, everything in 64 bits, the chosen experts given."""
    T, E, k = shape.T, shape.E, shape.k
    mu = h.mean(1, keepdim=True)
    c = h - mu
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    logits = y @ p["W_r"]
    sel = torch.gather(logits, 1, idx)
    w = torch.softmax(sel, 1)
    out = h
    for e in range(E):
        tok, j = (idx == e).nonzero(as_tuple=True)
        a = y[tok]
        z = torch.nn.functional.silu(a @ p["W_gate"][e]) * (a @ p["W_up"][e]) @ p["W_down"][e]
        out = out.index_add(0, tok, w[tok, j][:, None] * z)
    prob = torch.softmax(logits, 1).reshape(sequences, -1, E)
    hot = torch.nn.functional.one_hot(idx, E).sum(1).reshape(sequences, -1, E).double()
    f = hot.sum(1) / (hot.shape[1] * k)
    bal = (E * (f * prob.mean(1)).sum(1)).mean()
    z = torch.logsumexp(logits, 1).square().mean()
    return (out * d_out).sum() + g_balance * bal + g_z * z


def test_gradients_of_the_whole_block(ex):
    """bf16 rounds the activations between the operators (2^-9 each, about six in a row: 1e-2 of a gradient's size)."""
    shape = MoEShape(T=256, H=128, I=64, E=8, k=2)
    block = ex.Block(shape, sequences=2, g_balance=0.5, g_z=0.05, seed=5)
    x, r, target = ex.data(shape, ex.Block(shape, seed=6), 7)
    out = block.forward(x, r)
    d_out = ((out - target) / 16).to(torch.bfloat16).float()
    got = block.backward(d_out)
    assert block.status() == {}
    p = {n: w.to(torch.bfloat16).double().requires_grad_() for n, w in block.master.items()}
    h = block.normed["sum"].double().requires_grad_()
    loss = reference_loss(p, h, d_out.double(), block.layer.routing["topk_idx"].long(), shape, 2, 0.5, 0.05)
    loss.backward()
    ref = {"h": h.grad, **{n: t.grad for n, t in p.items()}}
    for n, t in ref.items():
        g = got[n].view(torch.bfloat16) if got[n].dtype == torch.int16 else got[n]
        rel = float(torch.linalg.vector_norm(g.double() - t) / torch.linalg.vector_norm(t))
        assert rel <= 2e-2, (n, rel)


def test_training_lowers_the_loss(ex):
    losses = ex.train(steps=40, log=None)
    first, last = sum(a for a, _ in losses[:5]) / 5, sum(a for a, _ in losses[-5:]) / 5
    assert last < 0.8 * first, (first, last)
    assert all(0.5 < b < 16 for _, b in losses)
