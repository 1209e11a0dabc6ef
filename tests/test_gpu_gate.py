"""The gate against a plain form in 64 bits: which experts (exactly), their weights, the dispatch indices, the gradient,
the bias' step.

Tolerances.  A weight is a ratio of exponentials: each expf is off by 2 ulp (2^-22 of itself) and, for the rounding of its
argument, by |argument| 2^-24; a sum of up to 16 (renormalised) or 256 terms (8 per lane, then 5 exchanges) by at most 16
roundings of 2^-24; quotients and the factor by 2 more.  In all (4 + 4 + 16 + 4 + range) 2^-24, range the logits' spread.
A gradient is such a weight times a difference of products that are at most |d| max: relative to the largest term it adds 8
roundings."""
import itertools

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape
from tests import gate_ref as R

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24


def rand(*s, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    return torch.randn(*s, generator=g, device="cuda")


def w_tolerance(logits):
    fine = logits[torch.isfinite(logits)]
    spread = float(fine.max() - fine.min()) if fine.numel() else 0.0
    return (28 + 2 * min(spread, 200.0)) * ULP


def check(logits, bias, k, flagged=False, renormalise=True, scale=1.0, score="sigmoid", **groups):
    T, E = logits.shape
    gate = moe.Gate(T, E, k, score=score, renormalise=renormalise, scale=scale, **groups)
    out = gate.forward(logits, bias=bias)
    assert gate.status() == {"forward": moe.DEV_NONFINITE_LOGIT if flagged else 0}
    clean = torch.where(torch.isnan(logits), torch.full_like(logits, -torch.inf), logits)
    clean = clean.clamp(max=torch.finfo(torch.float32).max)
    idx, has = R.choose(clean, bias, k, score, **groups)
    torch.testing.assert_close(out["topk_idx"].long(), idx, rtol=0, atol=0)
    w = R.weights(clean, idx, has, score, renormalise, scale)
    torch.testing.assert_close(out["topk_w"].double(), w, rtol=w_tolerance(clean), atol=scale * 2.0 ** -126)
    assert torch.all(out["topk_w"][~has] == 0)
    counts, offsets, rows, slots = R.dispatch(idx, E)
    for name, ref in (("counts", counts), ("offsets", offsets), ("row_of_slot", rows), ("slot_of_row", slots)):
        torch.testing.assert_close(out[name].long(), ref, rtol=0, atol=0, msg=name)
    torch.testing.assert_close(out["w_row"], out["topk_w"].reshape(-1)[slots], rtol=0, atol=0)
    return gate, out, idx, has


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (63, 16, 16), (65, 32, 4), (512, 8, 2), (513, 33, 6), (1000, 60, 4), (31, 256, 16),
         (577, 256, 1), (4099, 128, 8), (20011, 250, 6)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score,biased,renormalise", list(itertools.product(["softmax", "sigmoid"], [False, True],
                                                                            [False, True])))
def test_choice_and_weights(T, E, k, score, biased, renormalise):
    logits = rand(T, E, seed=T) + 0.7 * rand(E, seed=1)
    bias = torch.round(20 * rand(E, seed=2)) * 1e-3 if biased else None
    check(logits, bias, k, renormalise=renormalise, scale=2.5 if renormalise else 1.0, score=score)


@pytest.mark.parametrize("T,E,k,groups,top,best", [(1, 4, 2, 2, 1, 1), (300, 16, 4, 4, 2, 2), (65, 60, 6, 10, 3, 2),
                                                   (700, 64, 8, 32, 4, 2), (129, 160, 6, 8, 3, 1), (4097, 256, 8, 8, 4, 2),
                                                   (90, 32, 3, 32, 3, 1), (90, 96, 6, 3, 2, 2), (64, 250, 5, 5, 5, 2)])
@pytest.mark.parametrize("score,biased", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_groups(T, E, k, groups, top, best, score, biased):
    logits = rand(T, E, seed=T) * 1.5
    bias = 0.05 * rand(E, seed=2) if biased else None
    check(logits, bias, k, score=score, groups=groups, top_groups=top, group_best=best)


def test_a_large_batch():
    logits = rand(131072, 256)
    check(logits, torch.round(20 * rand(256, seed=2)) * 1e-3, 8, scale=2.5, groups=8, top_groups=4, group_best=2)


@pytest.mark.parametrize("E,k,biased", [(40, 8, True), (8, 2, False), (256, 1, True)])
def test_several_rounds_per_block(E, k, biased):
    """More tokens than the blocks take in one round, and more slots than the second kernel sorts at once."""
    check(rand(500003, E), 0.1 * rand(E) if biased else None, k)


@pytest.mark.parametrize("T", [255, 256, 257, 511, 512, 513, 4095, 19456, 19457, 194560, 194561])
def test_edges_of_chunks_and_clusters(T):
    check(rand(T, 16, seed=T), None, 3)


def test_rows_off_the_vectors_alignment():
    """Logits that start 16 and not 32 bytes off, for the widths that are otherwise read in whole sectors."""
    for E in (64, 128, 256):
        buf = rand(200 * E + 4)
        z = buf[4:].view(200, E)
        assert z.data_ptr() % 32 == 16
        check(z, 0.1 * rand(E, seed=1), 8)
        check(z, 0.1 * rand(E, seed=1), 8, groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("E,k,groups", [(8, 3, {}), (64, 6, {}), (256, 8, dict(groups=8, top_groups=3, group_best=2)),
                                        (96, 5, dict(groups=6, top_groups=2, group_best=1))])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("kind", ["zeros", "halves", "neighbours", "far", "tiny", "bf16"])
def test_ties_and_near_ties(E, k, groups, score, biased, kind):
    """Scores that are equal, or closer than fp32 holds: the order is the exact one, and equal ones go by index."""
    T = 200
    z = rand(T, E, seed=3)
    bias = torch.round(4 * rand(E, seed=4)) * 0.125 if biased else None
    if kind == "zeros":
        z.zero_()
    elif kind == "halves":
        z = torch.round(z * 2) / 2
    elif kind == "neighbours":  # a few units in the last place apart
        z = torch.full_like(z, 0.75) + torch.randint(0, 9, z.shape, device="cuda") * 2.0 ** -24
        if biased:
            bias = torch.randint(0, 9, (E,), device="cuda") * 2.0 ** -24
    elif kind == "far":  # sigmoids of 1 but for the last bits, and of nearly nothing
        z = torch.where(z > 0, 16 + z, -90 + 8 * z)
    elif kind == "tiny":
        z = -30 + z
        if biased:
            bias = torch.zeros_like(bias)
    else:
        z = z.to(torch.bfloat16).float()
    check(z, bias, k, score=score, **groups)


def test_signed_zeros_tie():
    z = torch.zeros(70, 40, device="cuda")
    z[:, ::2] = -0.0
    check(z, None, 7)


@pytest.mark.parametrize("groups", [{}, dict(groups=8, top_groups=3, group_best=2), dict(groups=8, top_groups=3, group_best=1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_experts_that_may_not_be_chosen(groups, score, biased, renormalise):
    T, E, k = 150, 64, 6
    z = rand(T, E, seed=5)
    z[rand(T, E, seed=6) > 0.3] = -torch.inf
    z[0] = -torch.inf                 # nothing is left
    z[1, 3:] = -torch.inf             # fewer than k
    z[2, :56] = -torch.inf            # one group
    z[3, torch.arange(E, device="cuda") % 8 != 0] = -torch.inf  # one expert in each group
    z[4] = torch.finfo(torch.float32).min
    bias = 0.1 * rand(E, seed=7) if biased else None
    check(z, bias, k, renormalise=renormalise, score=score, **groups)
    if biased:  # an expert that is off, and one that everybody takes
        bias[5], bias[9] = -torch.inf, torch.nan
        check(z, bias, k, renormalise=renormalise, score=score, **groups)
        bias[20] = torch.inf
        check(z, bias, k, renormalise=renormalise, score=score, **groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [100, 1500])
def test_logits_that_are_not_finite(score, T):
    z = rand(T, 40, seed=8)
    z[T // 2, 7] = torch.nan
    check(z, None, 4, flagged=True, score=score)
    z[3, 0] = torch.inf
    check(z, 0.1 * rand(40), 4, flagged=True, score=score)
    g = moe.Gate(T, 40, 4, score=score)
    g.forward(z)
    g.forward(rand(T, 40))
    assert g.status() == {"forward": 0}  # of the last call


def test_large_bias():
    """Far larger than the scores: fixed point holds nothing of these, the exact form does."""
    z = rand(300, 48, seed=9)
    bias = torch.zeros(48, device="cuda")
    bias[11], bias[3] = 1e6, -1e6
    check(z, bias, 4)


def test_no_tokens():
    g = moe.Gate(0, 16, 2)
    out = g.forward(torch.empty(0, 16, device="cuda"))
    assert int(out["counts"].abs().sum()) == 0 and int(out["offsets"].abs().sum()) == 0
    assert g.backward(torch.empty(0, 16, device="cuda"), out["topk_idx"], out["topk_w"], out["topk_w"]).shape == (0, 16)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (513, 33, 6), (31, 256, 16), (1001, 250, 3),
                                   (20000, 128, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_gradient(T, E, k, score, renormalise, masked):
    scale = 2.5
    z = rand(T, E, seed=10) * 2
    if masked:
        z[rand(T, E, seed=6) > 0.5] = -torch.inf
        z[0] = -torch.inf
    gate = moe.Gate(T, E, k, score=score, renormalise=renormalise, scale=scale)
    out = gate.forward(z)
    idx, has = R.choose(z, None, k, score)
    d = rand(T, k, seed=11)
    got = gate.backward(z, out["topk_idx"], out["topk_w"], d, d_logits=torch.full_like(z, 7.0))
    ref = R.gradient(z, idx, has, d, score, renormalise, scale)
    tol = (w_tolerance(z) + 24 * ULP) * scale * float(d.abs().max()) * 2
    torch.testing.assert_close(got.double(), ref, rtol=0, atol=tol)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_differences(score, renormalise):
    T, E, k, h = 20, 12, 3, 1e-5
    z, d = rand(T, E, seed=12), rand(T, k, seed=13).double()
    gate = moe.Gate(T, E, k, score=score, renormalise=renormalise, scale=1.5)
    out = gate.forward(z)
    got = gate.backward(z, out["topk_idx"], out["topk_w"], d.float())
    idx, has = R.choose(z, None, k, score)
    f = lambda l: (R.weights_of(l, idx, has, score, renormalise, 1.5) * d).sum(1)  # noqa: E731  (tokens are independent)
    for e in range(E):
        step = torch.zeros(E, device="cuda", dtype=torch.float64)
        step[e] = h
        diff = (f(z.double() + step) - f(z.double() - step)) / (2 * h)  # off by h^2 / 6 of the third derivative
        torch.testing.assert_close(got[:, e].double(), diff, rtol=0, atol=1e-5)


def test_gradient_of_bad_indices_has_no_part():
    z, d = rand(9, 8), rand(9, 2)
    gate = moe.Gate(9, 8, 2, score="sigmoid")
    out = gate.forward(z)
    idx = out["topk_idx"].clone()
    ref = gate.backward(z, idx, out["topk_w"], d)
    w = out["topk_w"].clone()
    w[4, 1] = 0
    ref = gate.backward(z, idx, w, d)
    idx[4, 1] = 99
    assert torch.equal(gate.backward(z, idx, out["topk_w"], d), ref)
    idx[4, 1] = -1
    assert torch.equal(gate.backward(z, idx, out["topk_w"], d), ref)


@pytest.mark.parametrize("rows,E", [(1, 8), (1, 256), (5, 33), (3000, 128)])
def test_bias_step(rows, E):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    counts = torch.randint(0, 50, (rows, E), generator=g, device="cuda", dtype=torch.int32)
    if E == 8:
        counts[0] = torch.tensor([4, 4, 4, 4, 5, 3, 4, 4])
    bias = rand(E)
    c = counts.long().sum(0)
    ref = bias + 0.25 * torch.sign(c.sum() - E * c)
    gate = moe.Gate(10, E, 1)
    gate.update_bias(bias, counts if rows > 1 else counts[0], 0.25)
    assert torch.equal(bias, ref)


def test_the_same_bits_every_time_and_in_a_graph():
    T, E, k = 5000, 128, 8
    a, b = rand(T, E), rand(T, E, seed=5)
    bias = 0.05 * rand(E)
    gate = moe.Gate(T, E, k, score="sigmoid")
    buf, out = a.clone(), None
    out = gate.forward(buf, bias)
    d = rand(T, k)
    grad = torch.empty_like(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gate.forward(buf, bias, out=out)
        gate.backward(buf, out["topk_idx"], out["topk_w"], d, d_logits=grad)
    for x in (a, b, a):
        buf.copy_(x)
        graph.replay()
        other = moe.Gate(T, E, k, score="sigmoid")
        ref = other.forward(x, bias)
        for n in ref:
            assert torch.equal(out[n], ref[n]), n
        assert torch.equal(grad, other.backward(x, ref["topk_idx"], ref["topk_w"], d))


def test_the_gate_agrees_with_the_layer_s_own_routing():
    """Softmax, renormalised, no bias: the same routing as the layer's own."""
    shape = MoEShape(T=3000, H=64, I=64, E=48, k=5)
    layer = moe.MoELayer(shape)
    z = rand(shape.T, shape.E)
    layer.route(z)
    out = moe.Gate(shape.T, shape.E, shape.k).forward(z)
    for n in ("topk_idx", "counts", "offsets", "row_of_slot", "slot_of_row"):
        assert torch.equal(out[n], layer.routing[n]), n
    torch.testing.assert_close(out["topk_w"], layer.routing["topk_w"], rtol=2 * w_tolerance(z), atol=0)
