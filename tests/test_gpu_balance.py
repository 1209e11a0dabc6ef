"""The balance loss and z loss with per-expert counts, and their gradient, against the formulas in 64 bits and
against differences.

Tolerances, from the arithmetic: expf and logf are good to 2 units in the last place and a softmax row sums at most
256 terms, so a probability is off by under 1e-6 of itself where |logits| < 20 (the argument's own rounding, 20 *
2^-24, is the largest part); sums over tokens add about sqrt of their depth.  Probabilities, losses and gradients
are held to 5e-6 of the largest of their kind.  Counts are whole numbers and equal."""
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


def make(T, E, k, seed, S=1, mask=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lg = torch.randn(T, E, generator=g, device="cuda") * 2 + torch.randn(E, generator=g, device="cuda")
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()
    m = None
    if mask == "random":
        m = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    elif mask == "padded":  # every sequence padded at its end, one of them empty
        L = T // S
        n = torch.randint(0, L + 1, (S,), generator=g, device="cuda")
        n[S // 2] = 0
        m = (torch.arange(L, device="cuda")[None] < n[:, None]).reshape(T).to(torch.uint8)
    elif mask == "none left":
        m = torch.zeros(T, dtype=torch.uint8, device="cuda")
    return lg, idx, m


def reference(lg, idx, m, E, k, S, g_bal=0.0, g_z=0.0):
    T = lg.shape[0]
    lg = lg.double()
    valid = torch.isfinite(lg).any(1) if T else torch.zeros(0, dtype=torch.bool, device="cuda")
    if m is not None:
        valid &= m.bool()
    safe = torch.where(valid[:, None], lg, torch.zeros_like(lg))
    p = torch.softmax(safe, 1) * valid[:, None]
    lse = torch.logsumexp(safe, 1)
    L = T // S
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    hot.scatter_add_(1, idx.long(), valid.double()[:, None].expand(T, k).contiguous())
    c = hot.reshape(S, L, E).sum(1)
    n = valid.double().reshape(S, L).sum(1)
    P = p.reshape(S, L, E).sum(1) / n.clamp(min=1)[:, None]
    f = c / (k * n.clamp(min=1))[:, None]
    used, N = float((n > 0).sum()), float(n.sum())
    bal = float(E * (f * P).sum()) / max(used, 1)
    z = float((lse ** 2 * valid).sum()) / max(N, 1)
    w = (g_bal * E / (max(used, 1) * n.clamp(min=1)))[:, None]
    dp = (w * f).repeat_interleave(L, 0) if L else torch.zeros(0, E, dtype=torch.float64, device="cuda")
    d = p * (dp - (p * dp).sum(1, keepdim=True)) + (2 * g_z / max(N, 1)) * (lse * valid)[:, None] * p
    return {"loss": (bal, z), "counts": c.to(torch.int32), "probs": P, "tokens": n.to(torch.int32),
            "lse": torch.where(valid, lse, torch.full_like(lse, math.inf)), "d": d}


def near(name, got, ref, tol=TOL):
    if got.numel():
        scale = float(ref.abs().max())
        err = float((got.double() - ref).abs().max())
        assert err <= tol * scale + 1e-30, (name, err, scale)


def check(T, E, k, S=1, mask=None, seed=1, edit=None):
    lg, idx, m = make(T, E, k, seed, S, mask)
    if edit:
        edit(lg, idx, m)
    b = moe.BalanceLoss(T, E, k, sequences=S)
    out = b.forward(lg, idx, mask=m)
    again = b.forward(lg, idx, mask=m)
    torch.cuda.synchronize()
    assert b.status() == {"forward": 0}
    r = reference(lg, idx, m, E, k, S, 0.3, 0.05)
    assert torch.equal(out["counts"], r["counts"]) and torch.equal(out["tokens"], r["tokens"])
    near("probs", out["probs"], r["probs"])
    assert torch.equal(torch.isinf(out["lse"]), torch.isinf(r["lse"]))
    fin = torch.isfinite(r["lse"])
    near("lse", out["lse"][fin], r["lse"][fin])
    for got, ref in zip(out["loss"].tolist(), r["loss"]):
        assert abs(got - ref) <= TOL * abs(ref) + 1e-30, (got, ref)
    assert all(torch.equal(out[n], again[n]) for n in out)
    d = b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.3, 0.05)
    near("d_logits", d, r["d"])
    old = torch.randn(T, E, device="cuda") * 1e-3
    acc = old.clone()
    b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.3, 0.05, d_logits=acc)
    near("d_logits added", acc, old.double() + r["d"])
    return lg, idx, m, out, d


# one token and one expert; every lane layout: whole vectors of 4 (E 4, 8, 60, 128, 132, 256) and single columns
# (E 1, 5, 31, 33, 65, 130, 255); token counts around a warp's, a block's and the grid's
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 4, 4), (100, 5, 2), (513, 8, 2), (333, 31, 3),
                                   (64, 33, 1), (999, 60, 4), (450, 65, 6), (4097, 128, 8), (777, 130, 7),
                                   (600, 132, 16), (2048, 255, 8), (20000, 256, 8)])
@pytest.mark.parametrize("mask", [None, "random"])
def test_sizes(T, E, k, mask):
    check(T, E, k, mask=mask)


@pytest.mark.parametrize("S,L", [(1, 1), (4, 1), (3, 50), (8, 640), (400, 3), (2, 9000)])
@pytest.mark.parametrize("mask", [None, "padded"])
def test_sequences(S, L, mask):
    check(S * L, 64, 4, S=S, mask=mask, seed=3)


def test_nothing_left_and_no_tokens():
    lg, idx, m, out, d = check(300, 16, 2, S=3, mask="none left")
    assert out["loss"].tolist() == [0.0, 0.0] and float(d.abs().max()) == 0
    _, _, _, out, _ = check(0, 16, 2, S=2)
    assert out["loss"].tolist() == [0.0, 0.0] and int(out["counts"].abs().sum()) == 0


def test_forbidden_experts_and_empty_rows():
    """-inf and the type's lowest value for experts that may not be chosen; rows that are -inf throughout."""
    def edit(lg, idx, m):
        lg[:, 3] = -math.inf
        lg[5:50, 7] = torch.finfo(torch.float32).min
        lg[10] = -math.inf
        lg[99] = -math.inf
        lg[20, 1:] = -math.inf
    lg, idx, m, out, d = check(100, 24, 2, edit=edit)
    assert float(d[:, 3].abs().max()) == 0 and float(d[10].abs().max()) == 0
    assert int(out["tokens"][0]) == 98


def test_garbage_in_padding_has_no_part():
    lg, idx, m = make(500, 40, 3, 8, 1, "random")
    b = moe.BalanceLoss(500, 40, 3)
    want = b.forward(lg, idx, mask=m)
    gone = m == 0
    lg2, idx2 = lg.clone(), idx.clone()
    lg2[gone] = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device="cuda").repeat(10)
    idx2[gone] = -12345
    got = b.forward(lg2, idx2, mask=m)
    assert b.status() == {"forward": 0}
    assert all(torch.equal(got[n], want[n]) for n in want)
    d = b.backward(lg2, got["counts"], got["tokens"], got["lse"], 1.0, 1.0)
    assert float(d[gone].abs().max()) == 0 and bool(torch.isfinite(d).all())
    acc = torch.full_like(lg, 2.0)
    b.backward(lg2, got["counts"], got["tokens"], got["lse"], 1.0, 1.0, d_logits=acc)
    assert bool((acc[gone] == 2.0).all())


def test_bad_values_are_reported():
    lg, idx, _ = make(200, 16, 2, 9)
    b = moe.BalanceLoss(200, 16, 2)
    bad = lg.clone()
    bad[3, 4] = math.nan
    out = b.forward(bad, idx)
    assert b.status()["forward"] == moe.DEV_NONFINITE_LOGIT and bool(torch.isnan(out["loss"]).all())
    wrong = idx.clone()
    wrong[0, 0], wrong[1, 1] = 16, -1
    out = b.forward(lg, wrong)
    assert b.status()["forward"] == moe.DEV_BAD_INDEX and int(out["counts"].sum()) == 398
    b.forward(lg, idx)
    assert b.status()["forward"] == 0


def test_even_load_gives_one():
    T, E, k = 256, 16, 2
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 1) % E], 1).to(torch.int32).cuda()
    out = moe.BalanceLoss(T, E, k).forward(torch.zeros(T, E, device="cuda"), idx)
    assert abs(float(out["loss"][0]) - 1) < 1e-6 and abs(float(out["loss"][1]) - math.log(E) ** 2) < 1e-5


@pytest.mark.parametrize("g_bal,g_z", [(1.0, 0.0), (0.0, 1.0)])
def test_gradient_against_differences(g_bal, g_z):
    """<d, v> against central differences of the loss in 64 bits with the counts held: the differences are good to
    step^2 = 1e-8 of the loss's third derivatives, the kernel's gradient to TOL of its size."""
    T, E, k, S = 60, 12, 3, 3
    lg, idx, m, out, _ = check(T, E, k, S=S, mask="random", seed=12)
    b = moe.BalanceLoss(T, E, k, sequences=S)
    d = b.backward(lg, out["counts"], out["tokens"], out["lse"], g_bal, g_z).double()
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    v = torch.randn(T, E, generator=g, device="cuda", dtype=torch.float64)
    step = 1e-4

    def loss(x):
        r = reference(x, idx, m, E, k, S)
        return g_bal * r["loss"][0] + g_z * r["loss"][1]
    diff = (loss(lg.double() + step * v) - loss(lg.double() - step * v)) / (2 * step)
    got = float((d * v).sum())
    assert abs(got - diff) <= 2e-5 * float((d * v).abs().sum()), (got, diff)


def test_counts_agree_with_the_router():
    """With one sequence and no padding the counts are moe_route's."""
    from dropless_mixture_experts_top_gb300.synth import MoEShape
    shape = MoEShape(T=1500, H=128, I=64, E=32, k=4)
    lg = make(1500, 32, 4, 14)[0]
    layer = moe.MoELayer(shape)
    layer.route(lg)
    out = moe.BalanceLoss(1500, 32, 4).forward(lg, layer.routing["topk_idx"])
    assert torch.equal(out["counts"][0], layer.routing["counts"])


def test_stream_and_graph():
    lg, idx, m = make(3000, 64, 4, 15, 4, "padded")
    b = moe.BalanceLoss(3000, 64, 4, sequences=4)
    out = b.forward(lg, idx, mask=m)
    d = b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.1, 0.1)
    want = {n: t.clone() for n, t in out.items()}, d.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = b.forward(lg, idx, mask=m, stream=s)
    s.synchronize()
    assert all(torch.equal(other[n], want[0][n]) for n in other)
    graph = torch.cuda.CUDAGraph()
    acc = torch.zeros_like(d)
    with torch.cuda.graph(graph):
        b.forward(lg, idx, mask=m, out=out)
        b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.1, 0.1, d_logits=acc)
    acc.zero_()
    for t in out.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[0][n]) for n in out) and torch.equal(acc, want[1])


def test_arguments_are_checked():
    lg, idx, _ = make(64, 8, 2, 16)
    b = moe.BalanceLoss(64, 8, 2)
    for kw in (dict(logits=lg[:32]), dict(logits=lg.half()), dict(logits=lg.cpu()), dict(topk_idx=idx.long()),
               dict(mask=torch.ones(63, dtype=torch.uint8, device="cuda")),
               dict(logits=torch.empty(8, 64, device="cuda").t())):
        with pytest.raises(ValueError):
            b.forward(**{**dict(logits=lg, topk_idx=idx), **kw})


def test_status_is_clear_before_the_first_call():
    size = moe.BalanceLoss(512, 8, 2, 1).fwd_scratch.numel()
    used = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    del used  # the allocator hands the same memory out again
    assert moe.BalanceLoss(512, 8, 2, 1).status() == {"forward": 0}


def test_more_logits_than_32_bits_count():
    """Two sequences whose logits pass the 2^31st element: rows there and the last ones, and whole counts."""
    E, k, base = 256, 2, 4096
    T = 2 ** 31 // E + 2 * base
    part, idx, _ = make(base, E, k, 12)
    lg, ix = part.repeat(T // base, 1), idx.repeat(T // base, 1)
    b = moe.BalanceLoss(T, E, k, sequences=2)
    out = b.forward(lg, ix)
    assert b.status() == {"forward": 0} and out["tokens"].tolist() == [T // 2, T // 2]
    counts = torch.bincount(idx.flatten().long(), minlength=E) * (T // base // 2)
    assert torch.equal(out["counts"].long(), counts.expand(2, E))
    r = reference(part, idx, None, E, k, 1, 0.3, 0.05)
    for at in (0, 2 ** 31 // E - base, 2 ** 31 // E, T - base):  # the same rows everywhere
        near("lse", out["lse"][at:at + base], r["lse"])
    d = b.backward(lg, out["counts"], out["tokens"], out["lse"], 0.3, 0.05, d_logits=None)
    # the gradient of the mean over all tokens is that of the part's mean, spread over T / base copies
    for at in (0, 2 ** 31 // E - base, 2 ** 31 // E, T - base):
        near("d_logits", d[at:at + base] * (T // base), r["d"])
