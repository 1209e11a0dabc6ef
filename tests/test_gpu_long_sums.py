"""The sums over all rows or tokens where there are more than 2^31 elements: the norm's weight gradients, the balance
loss, its z loss and mean probabilities, against 64-bit sums of a part that is repeated.

Tolerances, from the arithmetic.  A thread adds the terms of its rows one after another in fp32, n of them (900 rows
here, 1200 tokens), and the partial sums of threads and blocks meet in a tree of depth below 16.  Rounding n additions
of terms of one sign moves the sum by at most n 2^-24 / 2 of itself if every rounding falls the same way: 900 terms
2.7e-5, 1200 3.6e-5; roundings that fall either way leave about 1 / sqrt(n) of that, 1e-6.  Held to 2e-5 of the sum of
the terms' sizes (a twentieth of what a sum in 16 bits, or one that lost a thousandth of its rows, would show)."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu

TOL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("H", [8192, 8189])
def test_weight_gradients(kind, H):
    base = 1500
    T = (2 ** 31 // H + 3000) // base * base
    gen = torch.Generator(device="cuda")
    gen.manual_seed(81)
    x, dy = ((torch.randn(base, H, generator=gen, device="cuda") + 0.5).to(torch.bfloat16) for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(torch.bfloat16)
    n = moe.Norm(base, H, kind=kind)
    st = n.forward(x, w, w)["stats"]
    d, s = dy.double(), st.double()
    terms = d * (x.double() - s[:, :1]) * s[:, 1:]
    big = moe.Norm(T, H, kind=kind)
    r = T // base
    assert T * H > 2 ** 31
    g = big.backward(dy.repeat(r, 1), x.repeat(r, 1), w, st.repeat(r, 1))
    for name, t in (("dweight", terms), ("dbias", d)):
        over = (g[name].double() - r * t.sum(0)).abs() - TOL * r * t.abs().sum(0)
        assert float(over.max()) <= 0, name


@pytest.mark.parametrize("sequences", [1, 2])
def test_losses(sequences):
    E, k, base = 256, 2, 4096
    T = 2 ** 31 // E + 2 * base
    r = T // base
    assert T % (sequences * base) == 0 and T * E > 2 ** 31
    gen = torch.Generator(device="cuda")
    gen.manual_seed(82)
    lg = torch.randn(base, E, generator=gen, device="cuda") * 2
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32)
    out = moe.BalanceLoss(T, E, k, sequences=sequences).forward(lg.repeat(r, 1), idx.repeat(r, 1))
    P = torch.softmax(lg.double(), 1).mean(0)
    f = torch.bincount(idx.flatten().long(), minlength=E).double() / (base * k)
    assert float(((out["probs"].double() - P).abs() - TOL * P).max()) <= 0
    want = float(E * (f * P).sum()), float(torch.logsumexp(lg.double(), 1).square().mean())
    for got, ref in zip(out["loss"].tolist(), want):
        assert abs(got - ref) <= TOL * ref, (got, ref)
