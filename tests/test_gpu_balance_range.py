"""The balance loss and its gradient where logits are large and sequences are many.

Tolerance, from the arithmetic: a row's largest logits lie within 20 of its log sum here, whatever is added to all of
them, and two fp32 numbers of like size differ exactly.  exp is 2^(d log2 e) by the part's exponential (2 units in
the last place, 2.4e-7) of a rounded product (d log2 e <= 29, off by 2^-24 of itself: 1.2e-6 of the result); a row
sums at most 256 of them.  Together under 2e-6; probabilities and gradients are held to 5e-6 of the largest."""
import math

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu

TOL = 5e-6


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


def make(T, E, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lg = torch.randn(T, E, generator=g, device="cuda") * 2
    return lg, torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()


def reference(lg, idx, k, S, g_bal, g_z=0.0):
    """The gradient for logits, and P, of S sequences of unmasked tokens, in 64 bits."""
    T, E = lg.shape
    p = torch.softmax(lg.double(), 1)
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(
        1, idx.long(), torch.ones(T, k, dtype=torch.float64, device="cuda"))
    f = hot.reshape(S, T // S, E).mean(1) / k
    dp = (g_bal * E / T * f).repeat_interleave(T // S, 0)
    d = p * (dp - (p * dp).sum(1, keepdim=True)) + 2 * g_z / T * torch.logsumexp(lg.double(), 1)[:, None] * p
    return d, p.reshape(S, T // S, E).mean(1), f


def near(got, ref):
    assert bool(torch.isfinite(got).all())
    err, scale = float((got.double() - ref).abs().max()), float(ref.abs().max())
    assert err <= TOL * scale, (err, scale)


# every lane layout: whole vectors of 4 and more, of 2, single columns
@pytest.mark.parametrize("E,k", [(4, 2), (8, 2), (128, 8), (130, 6), (256, 8), (33, 2), (255, 8)])
@pytest.mark.parametrize("offset", [1e3, -1e4, 1e6, 1e30])
def test_a_common_offset_changes_nothing(E, k, offset):
    T, S = 300, 3
    lg, idx = make(T, E, k, 1)
    lg = lg + offset
    b = moe.BalanceLoss(T, E, k, sequences=S)
    out = b.forward(lg, idx)
    assert b.status() == {"forward": 0}
    d, P, f = reference(lg, idx, k, S, 0.5)
    near(out["probs"], P)
    near(b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.5, 0.0), d)
    old = torch.randn(T, E, device="cuda") * 1e-3
    acc = old.clone()
    b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.5, 0.0, d_logits=acc)
    near(acc, old.double() + d)


@pytest.mark.parametrize("E,k", [(8, 2), (128, 8), (130, 6), (33, 2)])
@pytest.mark.parametrize("value", [torch.finfo(torch.float32).min, -1e38, -1e9, 1e9, 1e38])
def test_rows_of_one_large_value(E, k, value):
    """Every expert is then as likely, also at the type's lowest value; rows beside them are not affected."""
    T = 96
    lg, idx = make(T, E, k, 2)
    lg[::3] = value
    b = moe.BalanceLoss(T, E, k)
    out = b.forward(lg, idx)
    d, P, _ = reference(lg, idx, k, 1, 1.0)
    near(out["probs"], P)
    got = b.backward(lg, out["counts"], out["tokens"], out["lse"], 1.0, 0.0)
    near(got, d)
    near(got[::3], d[::3])


def test_z_gradient_of_large_logits():
    T, E, k = 200, 64, 4
    lg, idx = make(T, E, k, 3)
    lg = lg + 5e3
    b = moe.BalanceLoss(T, E, k)
    out = b.forward(lg, idx)
    near(b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.0, 0.1), reference(lg, idx, k, 1, 0.0, 0.1)[0])


def test_many_sequences():
    """More sequences than blocks run at once, of one token and of a few."""
    for L, S, E, k in ((1, 5000, 8, 2), (3, 1700, 40, 4), (1, 1217, 256, 8), (300, 700, 5, 1),
                       (1, 40001, 8, 2), (2, 33333, 33, 4), (40, 32768, 4, 1), (1, 32769, 130, 3)):
        lg, idx = make(L * S, E, k, 4)
        b = moe.BalanceLoss(L * S, E, k, sequences=S)
        out = b.forward(lg, idx)
        d, P, f = reference(lg, idx, k, S, 0.5, 0.1)
        near(out["probs"], P)
        assert torch.equal(out["counts"], (f * k * L).round().int())
        assert bool((out["tokens"] == L).all())
        near(out["loss"][:1], (E * f * P).sum(1).mean()[None])
        near(b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.5, 0.1), d)
        old = torch.randn(L * S, E, device="cuda") * 1e-3
        acc = old.clone()
        b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.5, 0.1, d_logits=acc)
        near(acc, old.double() + d)


def test_the_backward_s_time_grows_with_the_sequences_alone():
    """Four times the sequences, one token each, take four times as long: less than eight, where each block going
    through every sequence would take sixteen."""
    def time(S):
        lg, idx = make(S, 8, 2, 5)
        b = moe.BalanceLoss(S, 8, 2, sequences=S)
        out = b.forward(lg, idx)
        d = torch.empty_like(lg)
        best = math.inf
        for _ in range(5):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            t0.record()
            b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.5, 0.1, d_logits=d)
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1))
        return best
    assert time(1 << 17) < 8 * time(1 << 15)
