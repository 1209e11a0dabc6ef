"""The orthogonalised update (Newton-Schulz products) against the same iteration in 64 bits.

Tolerances, from the arithmetic: rounding the result to bf16 alone is off by 1.7e-3 of it (2-norm, values spread evenly
between powers of two).  Each of five steps rounds X, S and P to fp16, 1.4e-4 of their size each, and what a step makes
of an error is at most 3.4 times it (its largest coefficient): sqrt(15) * 1.4e-4 * 3.4 = 1.9e-3 at most.  Together
2.5e-3; held to 4e-3.  Single values: the same noise within six deviations, 6 * 2.5e-3 < 3e-2 of the matrix's
root mean square, and bf16's last place, 2^-8 of the value."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu

REL, RMS = 4e-3, 3e-2


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


def grad(B, R, C, dtype, seed, scale=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(B, R, C, generator=g, device="cuda") * scale
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def reference(u, coefs, eps=1e-7, scale=1.0):
    x = u.double()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True).clamp(min=max(eps, 1e-300))
    for a, b, c in coefs:
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return scale * (x.transpose(1, 2) if tall else x)


def near(got, ref, rel=REL, rms=RMS):
    got = got.view(torch.bfloat16).double()
    assert got.shape == ref.shape and bool(torch.isfinite(got).all())
    if not got.numel():
        return
    for b in range(len(ref)):
        err, size = torch.linalg.vector_norm(got[b] - ref[b]), torch.linalg.vector_norm(ref[b])
        assert float(err) <= rel * float(size), (b, float(err / size))
        r = float(ref[b].pow(2).mean().sqrt())
        over = (got[b] - ref[b]).abs() - rms * r - 2.0 ** -8 * ref[b].abs()
        assert float(over.max()) <= 0, (b, float(over.max()) / r)


# one element, one row, one column; below, at and past a swizzle row (64), a CTA's rows (128), a tile (256), in both
# orientations; odd sizes; a long reduction; more matrices than CTA pairs
@pytest.mark.parametrize("B,R,C", [(1, 1, 1), (2, 1, 100), (2, 70, 1), (3, 8, 8), (2, 64, 64), (8, 128, 64),
                                   (2, 63, 65), (1, 128, 2048), (1, 2048, 128), (2, 256, 256), (2, 257, 300),
                                   (2, 300, 257), (3, 1000, 333), (2, 333, 1001), (1, 768, 520), (2, 512, 1536),
                                   (130, 64, 128), (80, 264, 328), (1, 1024, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sizes(B, R, C, dtype):
    g = grad(B, R, C, dtype, 1)
    o = moe.Orthogonaliser(B, R, C, dtype=dtype)
    out = o.update(g)
    assert o.status() == {"update": 0}
    near(out, reference(g, moe.MUON_COEFS))
    assert torch.equal(out, o.update(g))  # the same bits every time


# matrices that a cluster of CTAs holds on chip: 1 to 16 CTAs, ragged slabs, CTAs without columns, both orientations
@pytest.mark.parametrize("B,R,C", [(1, 128, 4096), (2, 4096, 96), (3, 100, 3000), (2, 1100, 128), (5, 64, 264),
                                   (2, 520, 33), (300, 16, 40), (1, 2, 4096), (40, 128, 1024), (1, 4097, 128),
                                   (2, 129, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_narrow(B, R, C, dtype):
    g = grad(B, R, C, dtype, 31)
    m = grad(B, R, C, "fp32", 32)
    u = g.double() + 0.95 * (0.95 * m.double() + g.double())
    o = moe.Orthogonaliser(B, R, C, dtype=dtype)
    near(o.update(g), reference(g, moe.MUON_COEFS))
    near(o.update(g, momentum=m), reference(u, moe.MUON_COEFS))
    assert o.status() == {"update": 0}


# every kind of row of the result: whole sectors (C % 16), whole vectors (C % 8), neither; results, inputs and scratch
# that start on a multiple of 16 bytes and not of 32
@pytest.mark.parametrize("C", [304, 312, 315, 64])
@pytest.mark.parametrize("R", [200, 650])
@pytest.mark.parametrize("first", [16, 8])
def test_result_rows(R, C, first):
    n = 2 * R * C
    g = torch.zeros(n + first, device="cuda", dtype=torch.bfloat16)[first:].view(2, R, C)
    g.copy_(grad(2, R, C, "bf16", 42))
    m = torch.zeros(n + first // 2, device="cuda")[first // 2:].view(2, R, C)
    base = torch.full((first + n + 16,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = base[first:first + n].view(2, R, C)
    o = moe.Orthogonaliser(2, R, C)
    o.scratch = torch.empty(o.scratch.numel() + 2 * first, dtype=torch.uint8, device="cuda")[2 * first:]
    o._scratch = o.scratch.data_ptr()
    assert out.data_ptr() % 32 == 2 * first % 32 and o._scratch % 32 == 2 * first % 32
    o.update(g, out=out)
    near(out, reference(g, moe.MUON_COEFS))
    o.update(g, momentum=m, out=out)
    near(out, reference(g, moe.MUON_COEFS))
    assert o.status() == {"update": 0}
    assert bool((base[:first] == 7).all()) and bool((base[first + n:] == 7).all())


# long sides that split the Gram product's reduction over clusters of 2 to 8 CTAs, in both orientations
@pytest.mark.parametrize("B,R,C", [(1, 2200, 160), (2, 200, 3000), (3, 2501, 333), (1, 900, 2320), (7, 300, 2200)])
def test_long_reductions(B, R, C):
    g = grad(B, R, C, "bf16", 41)
    o = moe.Orthogonaliser(B, R, C)
    out = o.update(g)
    assert o.status() == {"update": 0}
    near(out, reference(g, moe.MUON_COEFS))
    assert torch.equal(out, o.update(g))


def test_singular_values_end_near_one():
    g = grad(2, 384, 700, "fp32", 2)
    s = torch.linalg.svdvals(moe.Orthogonaliser(2, 384, 700, dtype="fp32").update(g).float())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", [(192, 320), (321, 111), (64, 104)])
@pytest.mark.parametrize("nesterov", [False, True])
def test_momentum(dtype, R, C, nesterov):
    B, beta = 3, 0.9
    o = moe.Orthogonaliser(B, R, C, dtype=dtype)
    m = grad(B, R, C, "fp32", 3)
    for step in range(3):
        g = grad(B, R, C, dtype, 10 + step)
        ref_m = beta * m.double() + g.double()
        out = o.update(g, momentum=m, beta=beta, nesterov=nesterov)
        # one fused multiply-add: within a unit in the last place of the larger term
        assert float((m.double() - ref_m).abs().max()) <= 2.0 ** -23 * float(ref_m.abs().max())
        u = g.double() + beta * m.double() if nesterov else m.double()
        near(out, reference(u, moe.MUON_COEFS))


@pytest.mark.parametrize("coefs", [((3.4445, -4.7750, 2.0315),), ((1.5, -0.5, 0.0),) * 4,
                                   ((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375))])
def test_other_steps_and_scale(coefs):
    g = grad(2, 200, 456, "bf16", 4)
    near(moe.Orthogonaliser(2, 200, 456, coefs=coefs).update(g, scale=-0.37), reference(g, coefs, scale=-0.37))


def test_size_of_the_update_has_no_part():
    for scale in (1e-12, 1.0, 1e12):
        g = grad(1, 96, 160, "bf16", 5, scale)
        near(moe.Orthogonaliser(1, 96, 160, eps=0.0).update(g), reference(g, moe.MUON_COEFS, eps=0.0))


@pytest.mark.parametrize("R,C", [(256, 304), (203, 301)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_updates_of_uneven_size(R, C, dtype):
    """Matrices whose parts differ widely in size: rows of zeros, one large value among small ones, sizes that change
    by 1e8 on the way, momentum without a gradient and a gradient that cancels it."""
    g = grad(6, R, C, dtype, 33, 1.0)
    g[1, :, : C - 1] = 0                                   # one column
    g[2] *= 1e-9
    g[2, R // 2, C // 3] = 1e3                             # one value
    g[3, : R // 2] *= 1e-8
    g[4, ::3] = 0
    g[5] = 0
    ref = reference(g, moe.MUON_COEFS)
    o = moe.Orthogonaliser(6, R, C, dtype=dtype)
    out = o.update(g).view(torch.bfloat16).double()
    assert o.status() == {"update": 0} and float(out[5].abs().max()) == 0
    near(out[[0, 4]].to(torch.bfloat16), ref[[0, 4]])
    for b in (1, 2, 3):
        # rank one, or half of the singular values 1e-8 of the others: what is small against the norm has no more
        # than its absolute exactness, 2^-12 per rounding and step, grown by at most 3.4445 a step
        err = torch.linalg.matrix_norm(out[b] - ref[b], ord=2)
        assert float(err) <= 0.05, (b, float(err))
    m = grad(6, R, C, "fp32", 34, 10.0)
    m[0] = -m[0].abs() * 0 - g[0].float() / 0.95           # cancels but for the nesterov term
    u = g.double() + 0.95 * (0.95 * m.double() + g.double())
    out = o.update(g, momentum=m)
    near(out[[5]], reference(u[[5]], moe.MUON_COEFS))
    near(out[[4]], reference(u[[4]], moe.MUON_COEFS))
    near(out[[0]], reference(u[[0]], moe.MUON_COEFS))


def test_zeros_and_bad_matrices_stay_their_own():
    g = grad(5, 136, 200, "bf16", 6)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[4, 135, 199] = float("inf")
    for eps in (1e-7, 0.0):
        o = moe.Orthogonaliser(5, 136, 200, eps=eps)
        out = o.update(g).float()
        assert o.status() == {"update": moe.DEV_NONFINITE_UPDATE}
        assert float(out[1].abs().max()) == 0
        assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[4]).all())
        near(out[[0, 3]].to(torch.bfloat16), reference(g[[0, 3]], moe.MUON_COEFS))
    g = grad(5, 136, 200, "bf16", 6)
    o.update(g)
    assert o.status() == {"update": 0}  # nothing of the last call is left


@pytest.mark.parametrize("R,C", [(136, 200), (136, 201), (64, 200)])
@pytest.mark.parametrize("momentum", [False, True])
def test_an_infinity_beside_a_nan_is_reported(R, C, momentum):
    g = grad(3, R, C, "bf16", 9)
    g[1, 3, 4], g[1, 3, 6], g[1, 3, 5] = float("nan"), float("nan"), float("inf")
    o = moe.Orthogonaliser(3, R, C)
    out = o.update(g, momentum=torch.zeros(3, R, C, device="cuda") if momentum else None).float()
    assert o.status() == {"update": moe.DEV_NONFINITE_UPDATE}
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isfinite(out[[0, 2]]).all())


def test_nothing_past_a_matrix_is_read_or_written():
    """Matrices of odd sizes between guard values: the neighbours of out, g and momentum keep theirs, and NaNs around
    g have no part."""
    B, R, C, pad = 2, 77, 131, 64
    n = B * R * C
    g = grad(B, R, C, "fp32", 7)
    m0 = grad(B, R, C, "fp32", 8)
    gb = torch.full((n + 2 * pad,), float("nan"), device="cuda")
    mb = torch.full((n + 2 * pad,), float("nan"), device="cuda")
    ob = torch.full((n + 2 * pad,), 7.0, device="cuda", dtype=torch.bfloat16)
    gb[pad:pad + n], mb[pad:pad + n] = g.flatten(), m0.flatten()
    o = moe.Orthogonaliser(B, R, C, dtype="fp32")
    o.scratch.fill_(255)  # NaNs in the workspace
    o.update(gb[pad:pad + n].view(B, R, C), momentum=mb[pad:pad + n].view(B, R, C),
             out=ob[pad:pad + n].view(B, R, C))
    m = 0.95 * m0.double() + g.double()
    near(ob[pad:pad + n].view(B, R, C), reference(g.double() + 0.95 * m, moe.MUON_COEFS))
    assert bool((ob[:pad] == 7).all()) and bool((ob[pad + n:] == 7).all())
    assert bool(torch.isnan(mb[:pad]).all()) and bool(torch.isnan(mb[pad + n:]).all())


def test_no_matrices():
    o = moe.Orthogonaliser(0, 64, 64)
    assert o.update(torch.empty(0, 64, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64, 64)
    assert o.status() == {"update": 0}


def test_int16_views_stream_and_graph():
    g = grad(3, 192, 256, "bf16", 9)
    o = moe.Orthogonaliser(3, 192, 256)
    want = o.update(g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = o.update(g.view(torch.int16), stream=s)
    s.synchronize()
    assert got.dtype == torch.int16 and torch.equal(got.view(torch.bfloat16), want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.update(g, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_two_streams():
    """Two objects on two streams at once give what each gives alone."""
    a, b = moe.Orthogonaliser(20, 256, 320), moe.Orthogonaliser(6, 640, 200)
    ga, gb = grad(20, 256, 320, "bf16", 20), grad(6, 640, 200, "bf16", 21)
    wa, wb = a.update(ga), b.update(gb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append((a.update(ga, stream=sa), b.update(gb, stream=sb)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in outs)


def test_arguments_are_checked():
    g = grad(2, 64, 96, "bf16", 12)
    o = moe.Orthogonaliser(2, 64, 96)
    m = torch.zeros(2, 64, 96, device="cuda")
    for kw in (dict(g=g[:1]), dict(g=g.float()), dict(g=g.cpu()), dict(g=g.transpose(1, 2)),
               dict(momentum=m.to(torch.bfloat16)), dict(momentum=m[:, :32]), dict(out=m)):
        with pytest.raises(ValueError):
            o.update(**{**dict(g=g), **kw})
    for coefs in ((), ((1.0, 2.0),)):
        with pytest.raises(ValueError):
            moe.Orthogonaliser(2, 64, 96, coefs=coefs)


def test_status_is_clear_before_the_first_call():
    size = moe.Orthogonaliser(2, 300, 200).scratch.numel()
    used = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    del used  # the allocator hands the same memory out again
    assert moe.Orthogonaliser(2, 300, 200).status() == {"update": 0}


@pytest.mark.parametrize("B,R,C", [(8200, 512, 512), (65535, 128, 264)])
def test_more_elements_than_32_bits_count(B, R, C):
    """Batches whose elements pass 2^31, in scratch and on chip: the first matrices, those there, and the last."""
    few = grad(9, R, C, "bf16", 13)
    g = few.repeat((B + 8) // 9, 1, 1)[:B].contiguous()
    o = moe.Orthogonaliser(B, R, C)
    out = o.update(g)
    assert o.status() == {"update": 0}
    cross = 2 ** 31 // (R * C)
    for b in (0, cross - 1, cross, cross + 1, B - 1):
        near(out[[b]], reference(g[[b]], moe.MUON_COEFS))


# enough work, and long enough sides, that two steps are taken at once: both orientations, whole and odd sizes, tiles of
# one CTA and of two; every number of steps up to five (an odd one by itself in the middle) and steps of other kinds
@pytest.mark.parametrize("B,R,C,steps", [(6, 600, 1500, 5), (6, 1507, 601, 5), (40, 300, 1100, 5), (2, 2100, 1024, 5),
                                         (6, 600, 1500, 1), (6, 1500, 600, 2), (6, 600, 1500, 3), (6, 1500, 600, 4)])
@pytest.mark.parametrize("mixed", [False, True])
def test_steps_in_pairs(B, R, C, steps, mixed):
    g, m = grad(B, R, C, "bf16", 51), grad(B, R, C, "fp32", 52)
    coefs = moe.MUON_COEFS[:steps]
    if mixed:
        coefs = [(1.5, -0.5, 0.0) if i % 2 else c for i, c in enumerate(coefs)]
    n, k = min(R, C), max(R, C)
    assert 4 * k >= 7 * n and 6 * n * n * (k - n) * B >= 1e10
    u = g.double() + 0.95 * (0.95 * m.double() + g.double())
    o = moe.Orthogonaliser(B, R, C, coefs=coefs)
    out = o.update(g, momentum=m)
    assert o.status() == {"update": 0}
    near(out, reference(u, coefs))
