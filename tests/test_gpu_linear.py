"""The dense layer against a plain form in 64 bits.

Where every input is a small whole number, all sums are exact in fp32 and the results have to be the exact ones rounded to
bf16, bit for bit.  Elsewhere: a bf16 rounding is off by 2^-8 of the value at most, 2^-8 / sqrt 3 in the mean square (2.3e-3);
the backward's products have one in dz, too (3.2e-3 together).  The fp32 sums' own error is at most n 2^-23 sum |terms| for n terms
(the tensor core may cut off instead of rounding)."""
import itertools
import math

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
RMS = 2.0 ** -8 / math.sqrt(3)
ACTS = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
        "gelu": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    return g


def whole(*s, seed=0, most=2):
    return torch.randint(-most, most + 1, s, generator=gen(seed), device="cuda").to(BF)


def randn(*s, seed=0, scale=1.0):
    return (torch.randn(*s, generator=gen(seed), device="cuda") * scale).to(BF)


# one row; ragged rows and columns; less than a tile; several; long reductions of few tiles (in parts); more tiles than a round
SIZES = [(1, 8, 8), (1, 64, 64), (2, 8, 4096), (3, 72, 40), (127, 128, 136), (129, 200, 264), (512, 128, 64), (777, 1000, 520),
         (300, 4096, 8), (1, 4096, 4096), (257, 5000, 2056), (2048, 64, 4096), (5000, 264, 1032), (30000, 128, 64),
         (4104, 1032, 4104), (16000, 520, 520), (2049, 1024, 4096), (2400, 264, 6144), (2300, 520, 4104)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("none", True, True), ("relu", True, False),
                                               ("relu", False, True)])
def test_forward_of_whole_numbers(T, K, N, act, bias, residual):
    x, W = whole(T, K, seed=1), whole(K, N, seed=2)
    b = whole(N, seed=3, most=9) if bias else None
    r = whole(T, N, seed=4, most=9) if residual else None
    lin = moe.Linear(T, K, N, activation=act, bias=bias)
    out = lin.forward(x, W, b, residual=r)
    assert lin.status() == {"last": 0}
    z = x.double() @ W.double()
    if bias:
        z = z + b.double()
    y = ACTS[act](z)
    if residual:
        y = y + r.double()
    assert torch.equal(out["y"], y.to(BF))
    if act == "none":
        assert out["z"] is None
    else:
        assert torch.equal(out["z"], z.to(BF))
        assert torch.equal(lin.forward(x, W, b, residual=r, save=False)["y"], out["y"])


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act,bias", [("none", False), ("none", True), ("relu", True)])
def test_backward_of_whole_numbers(T, K, N, act, bias):
    x, W, dy = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=5)
    z = whole(T, N, seed=6) if act != "none" else None
    lin = moe.Linear(T, K, N, activation=act, bias=bias)
    got = lin.backward(dy, x, W, z)
    assert lin.status() == {"last": 0}
    dz = dy.double() if z is None else dy.double() * (z > 0)
    assert torch.equal(got["dx"], (dz @ W.double().T).to(BF))
    assert torch.equal(got["dW"], (x.double().T @ dz).to(BF))
    if bias:
        assert torch.equal(got["dbias"].double(), dz.sum(0))
    else:
        assert got["dbias"] is None


def close(got, ref, rms, terms, n):
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all()
    if got.numel() >= 1000:
        assert float((got - ref).norm()) <= rms * float(ref.norm()) + 1e-30
    else:  # so few roundings need not average out: the result's is at most 2^-8 of it, those of dz 2^-8 of each term
        assert float((got - ref).norm()) <= 2.0 ** -8 * float(ref.norm() + 1.01 * terms.norm()) + 1e-30
    assert torch.all((got - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + n * 2.0 ** -23 * terms + rms * 8 * ref.abs().max())


@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (130, 72, 264), (777, 1000, 520), (2048, 768, 2048)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_real_numbers(T, K, N, act):
    x, W, b = randn(T, K, seed=1), randn(K, N, seed=2, scale=K ** -0.5), randn(N, seed=3)
    r, dy = randn(T, N, seed=4), randn(T, N, seed=5)
    lin = moe.Linear(T, K, N, activation=act)
    out = lin.forward(x, W, b, residual=r)
    z = x.double() @ W.double() + b.double()
    terms = x.double().abs() @ W.double().abs() + b.double().abs()
    close(out["y"], ACTS[act](z) + r.double(), RMS * 1.01, terms, K)
    if act != "none":
        close(out["z"], z, RMS * 1.01, terms, K)
    at = out["z"].double().requires_grad_() if act != "none" else None
    dz = dy.double() if at is None else torch.autograd.grad(ACTS[act](at), at, dy.double())[0]
    got = lin.backward(dy, x, W, out["z"])
    close(got["dx"], dz @ W.double().T, RMS * 1.5, dz.abs() @ W.double().abs().T, N)
    close(got["dW"], x.double().T @ dz, RMS * 1.5, x.double().abs().T @ dz.abs(), T)
    # the bias: fp32 sums (T / 2^24 of the terms) of slopes that are off by 2^-19 (the exponential's argument, at most 88, times 2^-24 and more)
    assert torch.all((got["dbias"].double() - dz.sum(0)).abs() <= (T * 2.0 ** -24 + 2.0 ** -19) * dy.double().abs().sum(0) * 1.2)


def every_bf16():
    b = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)
    return b[torch.isfinite(b)]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_every_value_through_the_activation(act):
    v = every_bf16()
    n = v.numel() // 8 * 8
    v = v[:n]
    lin = moe.Linear(1, 8, n, activation=act, bias=False)
    W = torch.zeros(8, n, device="cuda", dtype=BF)
    W[0] = v
    x = torch.zeros(1, 8, device="cuda", dtype=BF)
    x[0, 0] = 1
    out = lin.forward(x, W)
    assert torch.equal(out["z"][0], v) or torch.equal(out["z"][0].double(), v.double())  # (-0 + 0 is 0)
    ref = ACTS[act](v.double())
    if act == "gelu":  # (1 + tanh cancels in 64 bits, too, where little is left of it)
        ref = v.double() * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v.double() + 0.044715 * v.double() ** 3))
    # half a bf16 step; the exponential's 2^-14 of the value at the most (an argument of 88, gelu's after 5 roundings of 2^-24, one
    # more for the exponential's own product, and 2 ulp); a sigmoid
    # below fp32's smallest normal number is lost, which is 2^-126 |z| (and |z| < 104 where it is not zero anyway); half of
    # bf16's smallest step, 2^-134
    tol = (2.0 ** -8 + 2.0 ** -14) * ref.abs() + v.double().abs().clamp(max=104) * 2.0 ** -126 + 2.0 ** -134
    assert torch.all((out["y"][0].double() - ref).abs() <= tol)
    # the slope, by the bias' gradient of a single row
    one = torch.ones(1, n, device="cuda", dtype=BF)
    back = moe.Linear(1, 8, n, activation=act)
    got = back.backward(one, x, W, v.view(1, n), grads={"dx": None, "dW": None, "dbias": torch.empty(n, device="cuda")})
    at = v.double().clamp(-200, 200).requires_grad_()  # (beyond, 0 or 1 in 64 bits too)
    ref, = torch.autograd.grad(ACTS[act](at).sum(), at)
    # s, z s' and their sum: an exponential's error moves s by s (1 - s) times it, largest where the argument is about 1.5, and
    # z s' by |z| s (1 - s) times it: under 2^-18 each
    assert torch.all((got["dbias"].double() - ref).abs() <= 2.0 ** -16 * (1 + ref.abs()))
    # against differences
    h = 1e-4
    near = v.double()[(v.abs() < 30) & (v.abs() > 1e-3)]
    diff = (ACTS[act](near + h) - ACTS[act](near - h)) / (2 * h)
    assert torch.all((got["dbias"].double()[(v.abs() < 30) & (v.abs() > 1e-3)] - diff).abs() <= 2.0 ** -16 * 2 + 1e-7)


def test_single_gradients_and_reused_buffers():
    T, K, N = 300, 136, 200
    x, W, dy, z = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=3), whole(T, N, seed=4)
    lin = moe.Linear(T, K, N, activation="relu")
    full = lin.backward(dy, x, W, z)
    for keep in itertools.chain.from_iterable(itertools.combinations(("dx", "dW", "dbias"), r) for r in (1, 2)):
        g = {n: torch.full_like(full[n], 3) if n in keep else None for n in full}
        assert lin.backward(dy, x, W, z, grads=g) is g
        for n in keep:
            assert torch.equal(g[n], full[n]), (keep, n)
    none = moe.Linear(T, K, N, bias=False)
    full = none.backward(dy, x, W)
    for n in ("dx", "dW"):
        g = {"dx": None, "dW": None, "dbias": None, n: torch.empty_like(full[n])}
        assert torch.equal(none.backward(dy, x, W, grads=g)[n], full[n])


# few tiles: a reduction of two stages to many, whole, over clusters of 2, 4 and 8 (as many as run at once and more), in parts
@pytest.mark.parametrize("T,K,N", [(16, 136, 64), (16, 264, 1032), (130, 520, 264), (9, 1024, 1920), (9, 1024, 2056),
                                   (512, 1000, 1152), (513, 1000, 1152), (1216, 264, 1024), (1216, 264, 1032), (16, 16384, 64),
                                   (100, 8200, 392), (256, 5000, 1024)])
@pytest.mark.parametrize("residual", [False, True])
def test_few_tiles(T, K, N, residual):
    x, W, b = whole(T, K, seed=1), whole(K, N, seed=2), whole(N, seed=3, most=9)
    r = whole(T, N, seed=4, most=9) if residual else None
    lin = moe.Linear(T, K, N, activation="relu")
    out = lin.forward(x, W, b, residual=r)
    z = x.double() @ W.double() + b.double()
    assert torch.equal(out["z"], z.to(BF))
    assert torch.equal(out["y"], (z.clamp_min(0) + (r.double() if residual else 0)).to(BF))
    got = lin.backward(out["y"], x, W, out["z"])
    dz = out["y"].double() * (out["z"] > 0)
    assert lin.status() == {"last": 0}
    for n, ref, terms, depth in (("dx", dz @ W.double().T, dz.abs() @ W.double().abs().T, N),
                                 ("dW", x.double().T @ dz, x.double().abs().T @ dz.abs(), T)):
        # a rounding, and those of fp32 sums of `depth` terms, each exact
        assert torch.all((got[n].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + depth * 2.0 ** -24 * terms * 1.01)
    again = lin.forward(x, W, b, residual=r)
    assert torch.equal(again["y"], out["y"])
    assert all(torch.equal(v, got[k]) for k, v in lin.backward(out["y"], x, W, out["z"]).items() if v is not None)


# few tokens: one to eight and more, few and many columns, one row of eight to the longest reduction, runs that end inside
@pytest.mark.parametrize("K,N", [(8, 8), (8, 16), (16, 1032), (136, 1024), (1000, 72), (4096, 520), (1032, 4104), (65536, 8),
                                 (65528, 24), (8, 65536), (4096, 4096)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 9])
def test_few_tokens(T, K, N):
    x, W, b, r = whole(T, K, seed=1), whole(K, N, seed=2), whole(N, seed=3, most=9), whole(T, N, seed=4, most=9)
    z = x.double() @ W.double() + b.double()
    plain = moe.Linear(T, K, N, bias=False)
    assert torch.equal(plain.forward(x, W)["y"], (z - b.double()).to(BF))
    lin = moe.Linear(T, K, N, activation="relu")
    first = lin.forward(x, W, b, residual=r)
    assert lin.status() == {"last": 0}
    assert torch.equal(first["z"], z.to(BF)) and torch.equal(first["y"], (z.clamp_min(0) + r.double()).to(BF))
    ends = torch.full((T + 2, N), 7, device="cuda", dtype=BF)  # the rows around it stay as they were; over the residual
    ends[1:-1] = r
    lin.forward(x, W, b, residual=ends[1:-1], save=False, out={"y": ends[1:-1], "z": None})
    assert torch.equal(ends[1:-1], first["y"]) and bool((ends[0] == 7).all()) and bool((ends[-1] == 7).all())


@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_few_tokens_of_real_numbers(T, act):
    K, N = 1536, 1096
    x, W, b = randn(T, K, seed=1), randn(K, N, seed=2, scale=K ** -0.5), randn(N, seed=3)
    x[-1, 5] = float("nan")
    W[7, 9] = float("inf")
    out = moe.Linear(T, K, N, activation=act).forward(x, W, b)
    assert bool(out["y"][-1].isnan().all())
    if act == "none":
        assert not bool(out["y"][:, 9].isfinite().any())
    ok = [c for c in range(N) if c != 9]
    x, W = x[:-1], W[:, ok]
    z = x.double() @ W.double() + b[ok].double()
    terms = x.double().abs() @ W.double().abs() + b[ok].double().abs()
    if T > 1:
        close(out["y"][:-1, ok], ACTS[act](z), RMS * 1.01, terms, K)


# the two products in one launch or in two, of one round or more, whole or in parts
@pytest.mark.parametrize("T,K,N", [(1, 1024, 1024), (16, 1024, 1024), (100, 1536, 1408), (100, 1544, 1408), (2048, 512, 512),
                                   (3000, 384, 384), (8192, 128, 128), (9729, 128, 8), (64, 4096, 256), (1000, 264, 1000)])
def test_both_products_and_each_alone(T, K, N):
    x, W, dy = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=3)
    lin = moe.Linear(T, K, N, bias=False)
    full = lin.backward(dy, x, W)
    assert torch.equal(full["dx"], (dy.double() @ W.double().T).to(BF))
    assert torch.equal(full["dW"], (x.double().T @ dy.double()).to(BF))
    for n in ("dx", "dW"):
        g = {"dx": None, "dW": None, "dbias": None, n: torch.full_like(full[n], 3)}
        assert torch.equal(lin.backward(dy, x, W, grads=g)[n], full[n])
    assert lin.status() == {"last": 0}


def test_the_residual_in_place_and_int16_views():
    T, K, N = 700, 264, 392
    x, W, b, r = whole(T, K, seed=1), whole(K, N, seed=2), whole(N, seed=3), whole(T, N, seed=4)
    lin = moe.Linear(T, K, N)
    ref = lin.forward(x, W, b, residual=r)["y"]
    bits = [t.view(torch.int16) for t in (x, W, b, r)]
    out = lin.forward(*bits[:3], residual=bits[3])
    assert out["y"].dtype == torch.int16 and torch.equal(out["y"].view(BF), ref)
    y = r.clone()
    assert torch.equal(lin.forward(x, W, b, residual=y, out={"y": y, "z": None})["y"], ref)
    small = moe.Linear(1, 4096, 256)  # a product in parts
    x, W, b, r = whole(1, 4096), whole(4096, 256, seed=2), whole(256, seed=3), whole(1, 256, seed=4)
    ref = small.forward(x, W, b, residual=r)["y"]
    y = r.clone()
    assert torch.equal(small.forward(x, W, b, residual=y, out={"y": y, "z": None})["y"], ref)


def test_rows_that_start_on_sixteen_bytes_alone():
    """Tensors at an odd multiple of 16 bytes, and nothing written around them."""
    T, K, N = 200, 128, 160
    x, W, r = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=4)
    lin = moe.Linear(T, K, N, activation="relu", bias=False)
    ref = lin.forward(x, W, residual=r)

    def inside(t):
        buf = torch.full((t.numel() + 16,), 77.0, device="cuda", dtype=BF)
        buf[8:8 + t.numel()] = t.reshape(-1)
        return buf, buf[8:8 + t.numel()].view(t.shape)
    (_, x2), (_, W2), (_, r2) = inside(x), inside(W), inside(r)
    yb, y2 = inside(torch.zeros_like(ref["y"]))
    zb, z2 = inside(torch.zeros_like(ref["y"]))
    lin.forward(x2, W2, residual=r2, out={"y": y2, "z": z2})
    assert torch.equal(y2, ref["y"]) and torch.equal(z2, ref["z"])
    for b in (yb, zb):
        assert torch.all(b[:8] == 77) and torch.all(b[-8:] == 77)


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    T, K, N = 300, 136, 264
    x, W = whole(T, K, seed=1), whole(K, N, seed=2)
    lin = moe.Linear(T, K, N, bias=False)
    ref = lin.forward(x, W)["y"]
    x[17, 5] = torch.nan
    W[9, 33] = torch.inf
    out = lin.forward(x, W)["y"]
    rows, cols = torch.arange(T, device="cuda") != 17, torch.arange(N, device="cuda") != 33
    assert torch.equal(out[rows][:, cols], ref[rows][:, cols]) and torch.isnan(out[17]).all()
    assert not torch.isfinite(out[:, 33]).any()


def test_no_rows():
    lin = moe.Linear(0, 64, 72)
    e = lambda *s: torch.empty(*s, device="cuda", dtype=BF)  # noqa: E731
    assert lin.forward(e(0, 64), e(64, 72), e(72))["y"].shape == (0, 72)
    g = lin.backward(e(0, 72), e(0, 64), e(64, 72))
    assert not g["dW"].any() and not g["dbias"].any() and lin.status() == {"last": 0}


def test_two_plans_and_graphs():
    """A captured step replayed on new values gives what eager calls give; two captured graphs of one plan, too."""
    T, K, N = 900, 520, 264
    lin = moe.Linear(T, K, N, activation="gelu")
    x, W, b, dy = randn(T, K, seed=1), randn(K, N, seed=2, scale=0.05), randn(N, seed=3), randn(T, N, seed=4)
    out = lin.forward(x, W, b)
    grads = lin.backward(dy, x, W, out["z"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lin.forward(x, W, b, out=out)
            lin.backward(dy, x, W, out["z"], grads=grads)
        graphs.append(graph)
    for i in range(4):
        x.copy_(randn(T, K, seed=10 + i))
        graphs[i % 2].replay()
        other = moe.Linear(T, K, N, activation="gelu")
        ref = other.forward(x, W, b)
        assert all(torch.equal(out[n], ref[n]) for n in ref)
        ref = other.backward(dy, x, W, ref["z"])
        assert all(torch.equal(grads[n], ref[n]) for n in ref)


def test_layers_of_every_kind_in_one_graph():
    """One token, few tokens, clusters, parts and whole tiles one after another, each on what the last one wrote."""
    sizes = [(1, 512, 1024), (6, 264, 1032), (16, 2048, 512), (300, 4096, 136), (2048, 1024, 1280), (16, 16384, 64)]
    plans, calls = [], []
    for i, (T, K, N) in enumerate(sizes):
        a, b = moe.Linear(T, K, N, activation="relu", bias=False), moe.Linear(T, N, K, bias=False)
        x, W, V = whole(T, K, seed=i), whole(K, N, seed=20 + i, most=1), whole(N, K, seed=40 + i, most=1)
        first = a.forward(x, W)
        second = b.forward(first["y"], V, residual=x)
        g2 = b.backward(second["y"], first["y"], V)
        g1 = a.backward(g2["dx"], x, W, first["z"])
        plans.append((a, b))
        calls.append((x, W, V, first, second, g2, g1))

    def step():
        for (a, b), (x, W, V, first, second, g2, g1) in zip(plans, calls):
            a.forward(x, W, out=first)
            b.forward(first["y"], V, residual=x, out=second)
            b.backward(second["y"], first["y"], V, grads=g2)
            a.backward(g2["dx"], x, W, first["z"], grads=g1)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(3):
        for i, c in enumerate(calls):
            c[0].copy_(whole(*c[0].shape, seed=100 * turn + i))
        step()
        torch.cuda.synchronize()
        eager = [{k: v.clone() for d in c[3:] for k, v in d.items() if v is not None} for c in calls]
        for c in calls:
            for d in c[3:]:
                for v in d.values():
                    if v is not None:
                        v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for c, e in zip(calls, eager):
            last = {k: v for d in c[3:] for k, v in d.items() if v is not None}
            assert all(torch.equal(v, e[k]) for k, v in last.items())
            x, W, V, first, second, g2, g1 = c
            z = x.double() @ W.double()
            assert torch.equal(first["z"], z.to(BF)) and torch.equal(first["y"], z.to(BF).clamp_min(0))
            terms = first["y"].double() @ V.double().abs()
            ref = first["y"].double() @ V.double() + x.double()
            assert torch.all((second["y"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + V.shape[0] * 2.0 ** -24 * terms * 1.01)
    assert all(p.status() == {"last": 0} for ab in plans for p in ab)



# few tokens, whole tiles of single CTAs and of pairs, clusters, parts of both
PATHS = [(1, 1536, 1096), (8, 512, 520), (300, 136, 264), (2049, 1024, 4096), (16, 4096, 1536), (128, 30000, 64), (4104, 4104, 1032)]


@pytest.mark.parametrize("T,K,N", PATHS)
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_nan_passes_the_activation(T, K, N, act):
    x, W, b, r = whole(T, K, seed=1), whole(K, N, seed=2), whole(N, seed=3, most=9), whole(T, N, seed=4, most=9)
    lin = moe.Linear(T, K, N, activation=act)
    want = lin.forward(x, W, b, residual=r)
    bt = b.clone()
    bt[5] = torch.nan
    x[-1, K // 2] = torch.nan
    out = lin.forward(x, W, bt, residual=r)
    hit = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    hit[-1], hit[:, 5] = True, True
    for n in ("y", "z"):
        assert torch.equal(out[n].isnan(), hit)
        assert torch.equal(out[n][~hit], want[n][~hit])
    assert torch.equal(lin.forward(x, W, bt, residual=r, save=False)["y"].isnan(), hit)



@pytest.mark.parametrize("T,K,N", [(1, 64, 72), (777, 1000, 520), (2049, 1024, 4096)])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_nan_passes_the_slope(T, K, N, act):
    """A NaN of z is one of dz: its row of dx, its column of dW and its element of dbias, and nothing else."""
    x, W, dy, z = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=5), whole(T, N, seed=6)
    lin = moe.Linear(T, K, N, activation=act)
    z[-1, 9] = 0
    want = {n: t.clone() for n, t in lin.backward(dy, x, W, z).items()}
    z[-1, 9] = torch.nan
    got = lin.backward(dy, x, W, z)
    assert bool(got["dx"][-1].isnan().all()) and bool(got["dW"][:, 9].isnan().all()) and bool(got["dbias"][9].isnan())
    cols = torch.arange(N, device="cuda") != 9
    assert torch.equal(got["dx"][:-1], want["dx"][:-1])
    assert torch.equal(got["dW"][:, cols], want["dW"][:, cols]) and torch.equal(got["dbias"][cols], want["dbias"][cols])



@pytest.mark.parametrize("T,K,N", PATHS + [(1, 64, 72), (777, 1000, 520), (30000, 128, 64), (16000, 520, 520), (4104, 1032, 4104)])
def test_the_workspace_is_all_that_is_written(T, K, N):
    """Calls in a buffer that has 32 MB behind the workspace, as much as any product leaves in parts."""
    x, W, b, dy, z = whole(T, K, seed=1), whole(K, N, seed=2), whole(N, seed=3), whole(T, N, seed=5), whole(T, N, seed=6)
    lin = moe.Linear(T, K, N, activation="relu")
    want = lin.forward(x, W, b), lin.backward(dy, x, W, z)
    bwd = lin.scratch.numel()
    big = torch.full((bwd + (32 << 20),), 77, dtype=torch.uint8, device="cuda")
    lin.scratch, lin._scratch = big[:bwd], big.data_ptr()
    for size, call, ref in ((lin._fwd_bytes, lambda: lin.forward(x, W, b), want[0]),
                            (bwd, lambda: lin.backward(dy, x, W, z), want[1])):
        big.fill_(77)
        got = call()
        assert all(torch.equal(got[n], ref[n]) for n in ref)
        assert lin.status() == {"last": 0} and bool((big[size:] == 77).all())



def test_the_bias_alone_writes_no_dz():
    T, K, N = 3000, 64, 264
    x, W, dy, z = whole(T, K, seed=1), whole(K, N, seed=2), whole(T, N, seed=5), whole(T, N, seed=6)
    lin = moe.Linear(T, K, N, activation="relu")
    want = lin.backward(dy, x, W, z)["dbias"].clone()
    lin.scratch.fill_(77)
    got = lin.backward(dy, x, W, z, grads={"dx": None, "dW": None, "dbias": torch.empty(N, device="cuda")})
    assert torch.equal(got["dbias"], want) and lin.status() == {"last": 0}
    # the status word, and a partial row of dbias for every 96 rows
    assert int((lin.scratch != 77).sum()) <= 256 + -(-T // 96) * N * 4
