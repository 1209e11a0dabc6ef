"""The norm (layer and RMS kind) with its residual sum, and its backward, against the formulas in 64 bits and
against differences.

Tolerances, from the arithmetic: sums of up to 8192 fp32 terms in a tree of depth < 32 are off by at most about
32 * 2^-24 = 2e-6 of the terms' mean size, and a row whose mean is m deviations from zero loses m * 2^-24 more to the
subtraction (m <= 30 here: 2e-6); a normalised value or a gradient made of a few such sums is held to 2e-5 of the
row's largest one.  A bf16 output adds half a unit in the last place, 2^-9 of the value, held to 2^-8.  A column sum
over T rows in fp32 is held to 1e-5 of the sum of its terms' sizes."""
import numpy as np
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu

TOL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


def tensors(T, H, dtype, seed, offset=0.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    return {"x": (r(T, H) + offset).to(dt), "res": r(T, H).to(dt), "w": (1 + 0.2 * r(H)).to(dt),
            "b": (0.3 * r(H)).to(dt), "dy": r(T, H).to(dt), "ds": r(T, H).to(dt)}


def ref_forward(h, w, b, kind, eps):
    h, w = h.double(), w.double()
    mu = h.mean(1) if kind == "layer" else torch.zeros(len(h), dtype=torch.float64, device=h.device)
    c = h - mu[:, None]
    r = 1 / torch.sqrt((c * c).mean(1) + eps)
    y = c * r[:, None] * w
    return (y if b is None else y + b.double()), mu, r


def ref_backward(dy, h, w, mu, r, kind, ds):
    dy, h = dy.double(), h.double()
    xh = (h - mu[:, None]) * r[:, None]
    g = dy * w.double()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * r[:, None]
    return (dx if ds is None else dx + ds.double()), dy * xh, dy


def near_rows(name, got, ref, dtype):
    assert got.shape == ref.shape
    if not got.numel():
        return
    got = got.double()
    bound = TOL * ref.abs().amax(1, keepdim=True) + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0)
    over = (got - ref).abs() - bound
    assert torch.isfinite(got).all(), name
    assert float(over.max()) <= 1e-30, (name, float(over.max()))


def check(T, H, kind, dtype, bias, residual, seed=1, offset=0.5, eps=1e-5):
    t = tensors(T, H, dtype, seed, offset)
    n = moe.Norm(T, H, kind=kind, dtype=dtype, bias=bias, eps=eps)
    b, res, ds = (t["b"] if bias else None), (t["res"] if residual else None), (t["ds"] if residual else None)
    out = n.forward(t["x"], t["w"], b, residual=res)
    h = t["x"]
    if residual:
        h = (t["x"].float() + t["res"].float()).to(t["x"].dtype)
        assert torch.equal(out["sum"], h)
    else:
        assert out["sum"] is None
    y, mu, r = ref_forward(h, t["w"], b, kind, eps)
    near_rows("y", out["y"], y, dtype)
    if T:
        scale = h.double().abs().amax()
        assert float((out["stats"][:, 0].double() - mu).abs().max()) <= TOL * float(scale)
        assert float((out["stats"][:, 1].double() / r - 1).abs().max()) <= TOL
    g = n.backward(t["dy"], h, t["w"], out["stats"], d_sum=ds)
    again = n.backward(t["dy"], h, t["w"], out["stats"], d_sum=ds)
    # the backward is a function of the statistics it is given, in the 32 bits they are kept in
    dx, wt, bt = ref_backward(t["dy"], h, t["w"], out["stats"][:, 0].double(), out["stats"][:, 1].double(), kind, ds)
    near_rows("dx", g["dx"], dx, dtype)
    for name, terms in (("dweight", wt),) + ((("dbias", bt),) if bias else ()):
        err = (g[name].double() - terms.sum(0)).abs()
        assert float((err - 1e-5 * terms.abs().sum(0)).max()) <= 1e-30, (name, float(err.max()))
        assert torch.equal(g[name], again[name])
    assert bias or g["dbias"] is None
    return n, t, out, g


# one row and one element; rows below a vector, odd widths, widths of every thread count, the widest; row counts
# below, at and past a block's
@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (1, 7), (5, 8), (300, 64), (33, 100), (512, 128), (77, 129),
                                 (2500, 250), (700, 1000), (129, 2048), (1000, 2050), (310, 4096), (65, 5001),
                                 (64, 8192), (2, 8191)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sizes(T, H, dtype):
    check(T, H, "layer", dtype, True, True)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_forms(kind, dtype, bias, residual):
    check(401, 768, kind, dtype, bias, residual)
    check(17, 333, kind, dtype, bias, residual)


def test_no_rows():
    n, _, _, g = check(0, 256, "layer", "bf16", True, True)
    assert float(g["dweight"].abs().max()) == 0 and float(g["dbias"].abs().max()) == 0


def test_rows_far_from_zero_and_constant_rows():
    check(200, 1024, "layer", "fp32", True, False, offset=30.0)
    n = moe.Norm(4, 512, dtype="fp32", eps=1e-5)
    x = torch.full((4, 512), 3.0, device="cuda")
    w, b = torch.ones(512, device="cuda"), torch.full((512,), 0.25, device="cuda")
    out = n.forward(x, w, b)
    torch.cuda.synchronize()
    assert torch.equal(out["y"], torch.full_like(x, 0.25))  # zero deviation: the bias alone, no NaN


def test_a_bad_row_stays_its_own():
    t = tensors(64, 320, "bf16", 5)
    t["x"][7, 11] = float("nan")
    t["x"][9, 0] = float("inf")
    out = moe.Norm(64, 320).forward(t["x"], t["w"], t["b"])["y"]
    bad = ~torch.isfinite(out.float()).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 9]


def test_in_place_sum_and_gradient():
    """sum may be the residual itself, dx may be d_sum itself (the residual stream updated in place)."""
    t = tensors(333, 512, "bf16", 6)
    n = moe.Norm(333, 512)
    ref = n.forward(t["x"], t["w"], t["b"], residual=t["res"])
    g0 = n.backward(t["dy"], ref["sum"], t["w"], ref["stats"], d_sum=t["ds"])
    h, dh = t["res"].clone(), t["ds"].clone()
    out = n.forward(t["x"], t["w"], t["b"], residual=h,
                    out={"y": torch.empty_like(h), "sum": h, "stats": torch.empty_like(ref["stats"])})
    g = n.backward(t["dy"], h, t["w"], out["stats"], d_sum=dh,
                   grads={"dx": dh, "dweight": torch.empty_like(g0["dweight"]), "dbias": torch.empty_like(g0["dbias"])})
    assert torch.equal(h, ref["sum"]) and torch.equal(out["y"], ref["y"])
    assert torch.equal(dh, g0["dx"]) and torch.equal(g["dweight"], g0["dweight"])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(kind):
    """<dx, v>, <dw, v> and <db, v> against central differences of sum(y dy) in 64 bits: the difference's own error
    is of order step^2 = 1e-8, the kernel's fp32 gradients are good to TOL of their size."""
    n, t, out, g = check(37, 200, kind, "fp32", True, False, seed=9)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)

    def loss(x, w, b):
        return float((ref_forward(x, w, b, kind, 1e-5)[0] * t["dy"].double()).sum())
    arg = {"x": t["x"].double(), "w": t["w"].double(), "b": t["b"].double()}
    for name, grad in (("x", g["dx"]), ("w", g["dweight"]), ("b", g["dbias"])):
        v = torch.randn(arg[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        step = 1e-4
        up, dn = ({**arg, name: arg[name] + s * v} for s in (step, -step))
        diff = (loss(**up) - loss(**dn)) / (2 * step)
        got = float((grad.double() * v).sum())
        assert abs(got - diff) <= 1e-4 * float((grad.double() * v).abs().sum()), (name, got, diff)


def test_int16_views_and_stream_and_graph():
    t = tensors(300, 640, "bf16", 11)
    n = moe.Norm(300, 640)
    ref = n.forward(t["x"], t["w"], t["b"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = n.forward(t["x"].view(torch.int16), t["w"].view(torch.int16), t["b"].view(torch.int16), stream=s)
    s.synchronize()
    assert got["y"].dtype == torch.int16 and torch.equal(got["y"].view(torch.bfloat16), ref["y"])
    grads = n.backward(t["dy"], t["x"], t["w"], ref["stats"])
    want = {k: v.clone() for k, v in grads.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.forward(t["x"], t["w"], t["b"], out=ref)
        n.backward(t["dy"], t["x"], t["w"], ref["stats"], grads=grads)
    for v in grads.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(grads[k], want[k]) for k in want)


def test_arguments_are_checked():
    t = tensors(8, 64, "bf16", 12)
    n = moe.Norm(8, 64)
    for kw in (dict(x=t["x"][:4]), dict(x=t["x"].float()), dict(x=t["x"].cpu()), dict(weight=t["w"][:32]),
               dict(x=torch.empty(64, 8, dtype=torch.bfloat16, device="cuda").t()), dict(bias=None),
               dict(residual=t["res"][:, :32])):
        a = dict(x=t["x"], weight=t["w"], bias=t["b"])
        a.update(kw)
        with pytest.raises(ValueError):
            n.forward(**a)
    buf = torch.empty(8 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoEError) as e:  # 8 bytes past a 16-byte boundary
        n.forward(buf[4:].view(8, 64), t["w"], t["b"])
    assert e.value.code == -2


@pytest.mark.parametrize("H", [8192, 8189])
def test_more_elements_than_32_bits_count(H):
    """Rows before and after the 2^31st element, and the last ones, whole vectors and not."""
    T = 2 ** 31 // H + 3000
    t = tensors(1500, H, "bf16", 11)

    def longer(v):
        return v.repeat((T + 1499) // 1500, 1)[:T].contiguous()
    x, res, dy = longer(t["x"]), longer(t["res"]), longer(t["dy"])
    n = moe.Norm(T, H, kind="layer", dtype="bf16")
    out = n.forward(x, t["w"], t["b"], residual=res)
    g = n.backward(dy, out["sum"], t["w"], out["stats"], d_sum=res)
    cross = 2 ** 31 // H
    for r in (slice(0, 8), slice(cross - 8, cross + 8), slice(T - 8, T)):
        h = (x[r].float() + res[r].float()).to(torch.bfloat16)
        assert torch.equal(out["sum"][r], h)
        y, _, _ = ref_forward(h, t["w"], t["b"], "layer", 1e-5)
        near_rows("y", out["y"][r], y, "bf16")
        st = out["stats"][r].double()
        near_rows("dx", g["dx"][r], ref_backward(dy[r], h, t["w"], st[:, 0], st[:, 1], "layer", res[r])[0], "bf16")
