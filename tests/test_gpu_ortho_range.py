"""The orthogonalised update at the ends of its ranges: updates of any size, workspaces full of NaN, coefficients that
leave fp16's range.

Tolerances as derived for the update: bf16's rounding, 1.7e-3 of the result, and the fp16 roundings between products,
1.9e-3 at most: together 2.5e-3, held to 4e-3."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu

REL = 4e-3


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


def grad(B, R, C, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(B, R, C, generator=g, device="cuda") * scale
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def reference(u, coefs=moe.MUON_COEFS):
    x = u.double()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    for a, b, c in coefs:
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def near(got, ref):
    got = got.view(torch.bfloat16).double()
    assert bool(torch.isfinite(got).all())
    for b in range(len(ref)):
        err, size = torch.linalg.vector_norm(got[b] - ref[b]), torch.linalg.vector_norm(ref[b])
        assert float(err) <= REL * float(size), (b, float(err / size))


# in scratch: rows in vectors and single elements, both orientations, a split Gram product, steps in pairs; on chip
SIZES = [(2, 256, 304), (2, 203, 301), (2, 301, 203), (1, 200, 3000), (6, 600, 1500), (2, 96, 160), (2, 100, 252)]


@pytest.mark.parametrize("B,R,C", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-21, 1e-20, 1e-18, 1e-9, 1e9, 1e15])
def test_the_size_of_the_update_has_no_part(B, R, C, dtype, scale):
    """eps = 0, with and without momentum; the sum of the squares is inside fp32's range, the mean square (1e-42 at
    the least) need not be."""
    g, m = grad(B, R, C, dtype, 61, scale), grad(B, R, C, "fp32", 62, scale)
    o = moe.Orthogonaliser(B, R, C, dtype=dtype, eps=0.0)
    out = o.update(g)
    assert o.status() == {"update": 0}
    near(out, reference(g))
    u = g.double() + 0.95 * (0.95 * m.double() + g.double())
    out = o.update(g, momentum=m)
    assert o.status() == {"update": 0}
    near(out, reference(u))


@pytest.mark.parametrize("B,R,C", [(2, 256, 304), (2, 203, 301)])
def test_small_values_that_the_sample_misses(B, R, C):
    """No gradient, or one far smaller than the momentum, both tiny: X's first power of two is taken from the norm."""
    for scale in (0.0, 1e-30, 1e-24):
        g, m = grad(B, R, C, "fp32", 63, scale), grad(B, R, C, "fp32", 64, 1e-19)
        o = moe.Orthogonaliser(B, R, C, dtype="fp32", eps=0.0)
        u = g.double() + 0.95 * (0.95 * m.double() + g.double())
        out = o.update(g, momentum=m)
        assert o.status() == {"update": 0}
        near(out, reference(u))


# P past 65504 from a step on that finds s = 14; X past 255; the product of two steps' P past 65504 (steps in pairs)
@pytest.mark.parametrize("coefs", [((14.0, 0.0, 0.0), (3.4445, -4.7750, 2.0315)), ((400.0, 0.0, 0.0), (1.5, -0.5, 0.0)),
                                   ((1.0, 299.0, 0.0), (1.0, 0.01, 0.0))])
@pytest.mark.parametrize("B,R,C", [(2, 256, 304), (2, 301, 203), (6, 600, 1500), (6, 1500, 600), (2, 96, 160),
                                   (1, 128, 1000), (2, 100, 252), (2, 252, 100)])
def test_coefficients_that_leave_the_range_are_reported(coefs, B, R, C):
    """One value in a matrix is one singular value of 1.  The other matrices, of one value as well or of zeros, show
    that a finite result is not reported."""
    g = torch.zeros(B, R, C, device="cuda", dtype=torch.bfloat16)
    g[0, R // 2, C // 3] = 2.0
    o = moe.Orthogonaliser(B, R, C, coefs=coefs)
    out = o.update(g).float()
    assert o.status() == {"update": moe.DEV_NONFINITE_UPDATE}
    assert not bool(torch.isfinite(out[0]).all())
    assert B == 1 or float(out[1:].abs().max()) == 0
    # in range: the second P at 4647 and both together at 32529, and X at 200
    for fine in (((7.0, 0.0, 0.0), (3.4445, -4.7750, 2.0315)), ((200.0, 0.0, 0.0), (1.0, 0.0, 0.0))):
        o = moe.Orthogonaliser(B, R, C, coefs=fine)
        out = o.update(g)
        assert o.status() == {"update": 0}
        near(out[:1], reference(g[:1], fine))


# in scratch, where the padding of X, S and P is never written and read as zeros: both orientations, rows in vectors and
# single elements, a split Gram product, steps in pairs, a side just past a tile
@pytest.mark.parametrize("B,R,C", [(2, 203, 301), (2, 301, 203), (2, 129, 136), (1, 200, 3000), (1, 2501, 333),
                                   (6, 600, 1500), (6, 1507, 601), (2, 257, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nans_around_have_no_part(B, R, C, dtype):
    """A workspace full of NaN, NaN on either side of the gradient and the momentum, and guards around what is written."""
    pad, n = 64, B * R * C
    g, m0 = grad(B, R, C, dtype, 71), grad(B, R, C, "fp32", 72)
    gb = torch.full((n + 2 * pad,), float("nan"), device="cuda", dtype=g.dtype)
    mb = torch.full((n + 2 * pad,), float("nan"), device="cuda")
    ob = torch.full((n + 2 * pad,), 7.0, device="cuda", dtype=torch.bfloat16)
    gb[pad:pad + n], mb[pad:pad + n] = g.flatten(), m0.flatten()
    o = moe.Orthogonaliser(B, R, C, dtype=dtype)
    assert o.scratch.numel() > 4 * n  # the matrices are in it
    for momentum in (None, mb[pad:pad + n].view(B, R, C)):
        o.scratch.fill_(255)
        o.update(gb[pad:pad + n].view(B, R, C), momentum=momentum, out=ob[pad:pad + n].view(B, R, C))
        u = g.double()
        if momentum is not None:
            u = u + 0.95 * (0.95 * m0.double() + u)
        assert o.status() == {"update": 0}
        near(ob[pad:pad + n].view(B, R, C), reference(u))
    assert bool((ob[:pad] == 7).all()) and bool((ob[pad + n:] == 7).all())
    assert bool(torch.isnan(mb[:pad]).all()) and bool(torch.isnan(mb[pad + n:]).all())
    assert bool(torch.isnan(gb[:pad]).all()) and bool(torch.isnan(gb[pad + n:]).all())


@pytest.mark.parametrize("B,R,C", [(2, 256, 304), (2, 301, 203), (6, 600, 1500), (2, 96, 160), (2, 100, 252)])
@pytest.mark.parametrize("size", [1e-5, 1e-6])
def test_updates_below_eps(B, R, C, size):
    """u / eps then, and what the steps make of it; its values (times 256 in fp16) are above the subnormals."""
    eps = 1e-4
    g = grad(B, R, C, "fp32", 91, size * eps)
    x = g.double() / eps
    assert float(torch.linalg.vector_norm(g.double(), dim=(1, 2)).max()) < eps
    tall = R > C
    x = x.transpose(1, 2) if tall else x
    for a, b, c in moe.MUON_COEFS:
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    o = moe.Orthogonaliser(B, R, C, dtype="fp32", eps=eps)
    out = o.update(g)
    assert o.status() == {"update": 0}
    near(out, x.transpose(1, 2) if tall else x)
