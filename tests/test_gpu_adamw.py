"""The AdamW step over many tensors against the formulas in 64 bits.

Tolerances, in units of u = 2^-24 (half a step of fp32).  m and v: two products and a sum each, and for v the square: 4 u of the
largest term.  p: that error of m, through the update (where m's two terms cancel, it is more than any multiple of the update
itself: an m of b1 m + (1 - b1) g = 0 has an error of 4 u (1 - b1) |g| all the same, and the update is lr / corr1 / (root + eps)
times m); the update's factors (lr / corr1, 1 / root of corr2: 6 u each with their expm1 and log), root, sum and
quotient: 24 u of the update, and 2 u of p for its own product and sum.  bf16 parameters: half a step, 2^-8
(finfo.eps / 2), more.  8-bit states: half a step of e4m3, 2^-4 of the value or 2^-10 of the scale, with 8 u for the fp32 in front."""
import math

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
ODD = [(1,), (3,), (255,), (256,), (257,), (0,), (5, 7), (64, 64), (1000, 333), (2, 3, 129), (4097,)]


def rand(*s, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    return torch.randn(*s, generator=g, device="cuda") * scale


def offsets(shapes):
    at = [0]
    for s in shapes:
        at.append(at[-1] + -(-math.prod(s) // 256) * 256)
    return at


def held(state, bits):
    """m and v as the states hold them, in 64 bits."""
    if bits == 32:
        return state["m"].double(), state["v"].double()
    m, r = (state[n].double().view(-1, 256) * state[n + "_scale"].double()[:, None] for n in ("m", "v"))
    return m.reshape(-1), r.square().reshape(-1)


def reference(p, g, m, v, t, lr, decay, b1, b2, eps):
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    upd = lr / (1 - b1 ** t) * m / ((v / (1 - b2 ** t)).sqrt() + eps)
    return p * (1 - lr * decay) - upd, upd, m, v


def check_step(opt, shapes, params, grads, state, lr, decay, copies=None, scale=1.0, b1=0.9, b2=0.95, eps=1e-8, **kw):
    at, bits = offsets(shapes), opt.bits
    t = int(state["step"][1]) + 1
    m0, v0 = held(state, bits)
    before = {n: x.clone() for n, x in state.items()}
    old = [p.double() for p in params]
    opt.step(params, grads, state, kw.pop("lr_given", lr), copies=copies, **kw)
    assert opt.status(state) == {"step": 0} and state["step"].tolist() == [0, t, 0, 0]
    m1, v1 = held(state, bits)
    for i, s in enumerate(shapes):
        n, lo = math.prod(s), at[i]
        g = grads[i].double().reshape(-1) * scale
        p, upd, m, v = reference(old[i].reshape(-1), g, m0[lo:lo + n], v0[lo:lo + n], t, lr, decay[i], b1, b2, eps)
        got = params[i].double().reshape(-1)
        big_m = b1 * m0[lo:lo + n].abs() + (1 - b1) * g.abs()
        per_m = lr / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + eps)
        err = 4 * U * big_m * per_m + 24 * U * upd.abs() + 2 * U * (old[i].reshape(-1).abs() + upd.abs()) + 1e-37
        if params[i].dtype == torch.bfloat16:
            err = err + 2.0 ** -8 * (p.abs() + err)
        assert torch.all((got - p).abs() <= err), (i, s)
        if copies is not None and copies[i] is not None:
            assert torch.equal(copies[i], params[i].to(torch.bfloat16))
        if bits == 32:
            assert torch.all((m1[lo:lo + n] - m).abs() <= 4 * U * big_m + 1e-44), (i, s)
            assert torch.all((v1[lo:lo + n] - v).abs() <= 5 * U * v + 1e-44), (i, s)
        elif n:
            blk = torch.arange(lo, lo + n, device="cuda") // 256
            for name, exact, size in (("m", m, big_m), ("v", v.sqrt(), v.sqrt())):
                sc = state[name + "_scale"].double()[blk]
                most = torch.zeros_like(state["m_scale"], dtype=torch.float64).scatter_reduce_(0, blk, exact.abs(), "amax")
                torch.testing.assert_close(sc, most.clamp(min=1e-30)[blk] / 448, rtol=8 * U, atol=8 * U * float(size.max()) / 448)
                val = state[name].double()[lo:lo + n] * sc
                half = torch.maximum(exact.abs() * 2.0 ** -4, sc * 2.0 ** -10) + 8 * U * size
                if name == "v":
                    some = (exact > 0) & (v.float() > 0)
                    assert torch.all(val[some] > 0)
                    half = torch.where(exact < sc * 2.0 ** -9, sc * 2.0 ** -9, half)
                assert torch.all((val - exact).abs() <= half), (i, s, name)
        pad = slice(lo + n, at[i + 1])  # behind a tensor's end nothing changes
        for name in ("m", "v"):
            assert torch.equal(state[name].view(torch.uint8 if bits == 8 else torch.int32)[pad],
                               before[name].view(torch.uint8 if bits == 8 else torch.int32)[pad])


@pytest.mark.parametrize("param", ["fp32", "bf16"])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("bits", ["fp32", "8bit"])
def test_steps_of_odd_tensors(param, grad, bits):
    decay = [0.1 * (len(s) > 1) for s in ODD]
    opt = moe.AdamW(ODD, param=param, grad=grad, state=bits, weight_decay=decay, beta1=0.9, beta2=0.95)
    params = [rand(*s, seed=i).to(DT[param]) for i, s in enumerate(ODD)]
    copies = [p.to(torch.bfloat16) if i % 3 else None for i, p in enumerate(params)] if param == "fp32" else None
    state = opt.new_state()
    state["m"].view(torch.uint8).fill_(7)  # the padding, too: it is left alone
    state["m"].zero_() if bits == "fp32" else None
    if bits == "8bit":
        state["m"].view(torch.uint8).fill_(0)
    for t in range(4):
        grads = [(rand(*s, seed=100 * t + i) * torch.exp(3 * rand(*s, seed=7 + t))).to(DT[grad]) for i, s in enumerate(ODD)]
        check_step(opt, ODD, params, grads, state, 3e-3, decay, copies=copies)


@pytest.mark.parametrize("bits", ["fp32", "8bit"])
def test_many_tensors_are_several_launches(bits):
    shapes = [(1 + 37 * i % 700,) for i in range(150)] + [(0,)] * 70 + [(13, 11)]
    opt = moe.AdamW(shapes, state=bits, weight_decay=0.0, beta2=0.95)
    params = [rand(*s, seed=i) for i, s in enumerate(shapes)]
    state = opt.new_state()
    for t in range(3):
        grads = [rand(*s, seed=i + 1000 * t).to(torch.bfloat16) for i, s in enumerate(shapes)]
        check_step(opt, shapes, params, grads, state, 1e-2, [0.0] * len(shapes))


@pytest.mark.parametrize("bits", ["fp32", "8bit"])
def test_a_large_tensor(bits):
    shapes = [(128,), (40_000_003,), (128, 9)]
    opt = moe.AdamW(shapes, grad="fp32", state=bits, weight_decay=0.01, beta2=0.95)
    params = [rand(*s, seed=i) for i, s in enumerate(shapes)]
    state = opt.new_state()
    for t in range(2):
        check_step(opt, shapes, params, [rand(*s, seed=i + 10 * t) for i, s in enumerate(shapes)], state, 1e-2, [0.01] * 3)


@pytest.mark.parametrize("bits", ["fp32", "8bit"])
@pytest.mark.parametrize("b1,b2,eps", [(0.0, 0.0, 1e-8), (0.9, 0.999, 1e-3), (0.99, 0.9999, 1e-8)])
@pytest.mark.parametrize("done", [0, 1, 99, 2_000_000])
def test_betas_and_late_steps(bits, b1, b2, eps, done):
    shapes = [(700,), (3, 5)]
    opt = moe.AdamW(shapes, grad="fp32", state=bits, beta1=b1, beta2=b2, eps=eps, weight_decay=0.01)
    state = opt.new_state()
    state["step"][1] = done
    params = [rand(*s, seed=i) for i, s in enumerate(shapes)]
    check_step(opt, shapes, params, [rand(*s, seed=i + 5) for i, s in enumerate(shapes)], state, 1e-2, [0.01] * 2, b1=b1, b2=b2,
               eps=eps)


@pytest.mark.parametrize("bits", ["fp32", "8bit"])
def test_gradients_far_apart_and_zero(bits):
    """Within a block: zeros, tiny and large values; a root above zero is never held as zero."""
    shapes = [(512,), (256,), (300,)]
    opt = moe.AdamW(shapes, grad="fp32", state=bits, beta2=0.95, weight_decay=0.0)
    params, state = [rand(*s, seed=i) for i, s in enumerate(shapes)], opt.new_state()
    g = rand(512)
    g[:256] *= torch.logspace(-8, 3, 256, device="cuda")
    g[300:400] = 0
    for t in range(3):
        check_step(opt, shapes, params, [g * (1 + t), torch.zeros(256, device="cuda"), rand(300, scale=1e-12, seed=t)], state, 1e-3,
                   [0.0] * 3)
    assert torch.all(params[1] == rand(256, seed=1))  # no gradient, no decay: no change


def test_scale_and_rate_on_the_device():
    shapes = [(1000,), (64, 32)]
    opt = moe.AdamW(shapes, grad="fp32", beta2=0.95, weight_decay=0.1)
    params, state = [rand(*s, seed=i) for i, s in enumerate(shapes)], opt.new_state()
    lr, scale = torch.full((), 0.01, device="cuda"), torch.full((1,), 0.125, device="cuda")
    grads = [rand(*s, seed=i + 3) for i, s in enumerate(shapes)]
    check_step(opt, shapes, params, grads, state, float(lr), [0.1] * 2, scale=0.125, lr_given=lr, grad_scale=scale)
    kept = [p.clone() for p in params], {n: x.clone() for n, x in state.items()}
    for bad in (float("inf"), float("nan")):  # the step is left out
        scale.fill_(bad)
        opt.step(params, grads, state, 0.01, grad_scale=scale)
        assert opt.status(state) == {"step": moe.DEV_NONFINITE_UPDATE}
        assert all(torch.equal(a, b) for a, b in zip(params, kept[0]))
        assert all(torch.equal(state[n], kept[1][n]) for n in ("m", "v")) and state["step"].tolist()[1:] == [1, 0, 0]
    scale.fill_(0.125)
    check_step(opt, shapes, params, grads, state, float(lr), [0.1] * 2, scale=0.125, lr_given=lr, grad_scale=scale)


@pytest.mark.parametrize("bits", ["fp32", "8bit"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e30])
def test_a_gradient_that_is_not_finite_stays_where_it_is(bits, bad):
    shapes = [(600,)]
    opt = moe.AdamW(shapes, grad="fp32", state=bits, beta2=0.95)
    one, two = ([rand(600)], [rand(600)])
    st1, st2 = opt.new_state(), opt.new_state()
    g = rand(600, seed=4)
    h = g.clone()
    h[301] = bad
    opt.step(one, [g], st1, 1e-2)
    opt.step(two, [h], st2, 1e-2)
    assert opt.status(st1) == {"step": 0} and opt.status(st2) == {"step": moe.DEV_NONFINITE_UPDATE}
    rest = torch.arange(600, device="cuda") != 301
    assert torch.equal(one[0][rest], two[0][rest])
    if bad != 3e30:
        assert torch.isnan(two[0][301])
        far = torch.arange(600, device="cuda") // 256 != 1
        (_, v1), (_, v2) = held(st1, opt.bits), held(st2, opt.bits)
        assert torch.equal(v1[:600][rest], v2[:600][rest])
        assert torch.equal(v1[:600][far], v2[:600][far])


def test_captured_steps_count_on():
    shapes = [(300,), (17, 40)]
    opt = moe.AdamW(shapes, beta2=0.95, state="8bit")
    params, state = [rand(*s, seed=i) for i, s in enumerate(shapes)], opt.new_state()
    twin, tstate = [p.clone() for p in params], opt.new_state()
    grads = [rand(*s, seed=9).to(torch.bfloat16) for s in shapes]
    lr = torch.full((1,), 0.01, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        opt.step(params, grads, state, lr)
    for t in range(4):
        for i, g in enumerate(grads):
            g.copy_(rand(*shapes[i], seed=50 + t))
        lr.fill_(0.01 / (1 + t))
        graph.replay()
        opt.step(twin, grads, tstate, float(lr))
        assert all(torch.equal(a, b) for a, b in zip(params, twin))
        assert all(torch.equal(state[n].view(torch.uint8), tstate[n].view(torch.uint8)) for n in state)
    assert int(state["step"][1]) == 4


def test_no_tensors_and_empty_ones():
    for shapes in ([], [(0,), (0, 4)]):
        opt = moe.AdamW(shapes)
        state = opt.new_state()
        opt.step([torch.empty(s, device="cuda") for s in shapes],
                 [torch.empty(s, device="cuda", dtype=torch.bfloat16) for s in shapes], state, 0.1)
        assert state["step"].tolist() == [0, 1, 0, 0]


def test_against_a_long_plain_run():
    """Thirty steps of one tensor against the 64-bit recurrence: roundings of 30 steps, each as in a single one."""
    shapes = [(4000,)]
    opt = moe.AdamW(shapes, grad="fp32", beta2=0.95, weight_decay=0.1)
    p, state = rand(4000), opt.new_state()
    p64, m, v = p.double(), torch.zeros(4000, device="cuda", dtype=torch.float64), torch.zeros(4000, device="cuda", dtype=torch.float64)
    moved = torch.zeros_like(m)
    for t in range(1, 31):
        g = rand(4000, seed=t)
        opt.step([p], [g], state, 1e-2)
        p64, upd, m, v = reference(p64, g.double(), m, v, t, 1e-2, 0.1, 0.9, 0.95, 1e-8)
        moved += upd.abs()
    # m and v are off by at most 30 steps' roundings of their largest terms, relative to the root of v, which is of |g|'s size
    assert torch.all((p.double() - p64).abs() <= 30 * (2 * U * (p64.abs() + moved)) + 30 * 24 * U * (moved + 1e-2))



@pytest.mark.parametrize("bits", ["fp32", "8bit"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e20, 3e30, "parameter"])
def test_an_element_that_is_not_finite_leaves_its_block_alone(bits, bad):
    """The other elements' parameters, states and scales are those of a run in which the element has no gradient, in that
    step and in the next one; a gradient of 1e20 makes v infinite and m no more than large."""
    opt = moe.AdamW([(600,)], grad="fp32", state=bits, beta2=0.95)
    rest = torch.arange(600, device="cuda") != 301
    g = rand(600, seed=4)
    runs = []
    for odd in (False, True):
        p, state, h = rand(600), opt.new_state(), g.clone()
        h[301] = 0.0
        if odd and bad == "parameter":
            p[301], h[301] = float("inf"), 50.0  # m and v are finite, and the block's largest
        elif odd:
            h[301] = bad
        held_after = []
        for _ in range(2):
            opt.step([p], [h], state, 1e-2)
            assert opt.status(state) == {"step": moe.DEV_NONFINITE_UPDATE if odd else 0}
            held_after.append([p[rest]] + [state[n].view(torch.uint8 if bits == "8bit" else torch.int32)[:600][rest]
                                           for n in ("m", "v")] +
                              [state[n].clone() for n in ("m_scale", "v_scale") if n in state])
            h = rand(600, seed=5)
            h[301] = 0.0
        if odd and bits == "8bit":
            assert torch.isnan(state["m"].float()[301]) and torch.isnan(state["v"].float()[301])
        runs.append(held_after)
    for a, b in zip(*runs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))



@pytest.mark.parametrize("bits", ["fp32", "8bit"])
@pytest.mark.parametrize("param", ["fp32", "bf16"])
@pytest.mark.parametrize("step,infinite", [(3e35, False), (1e36, True)])
def test_a_parameter_that_rounds_to_infinity(bits, param, step, infinite):
    """bf16's largest, (2 - 2^-7) 2^127, moved by less and by more than half a step of it, 2^119 = 6.6e35; fp32 holds both."""
    opt = moe.AdamW([(300,)], param=param, grad="fp32", state=bits, weight_decay=0.0)
    p, g = torch.ones(300, device="cuda", dtype=DT[param]), torch.zeros(300, device="cuda")
    p[77], g[77] = torch.finfo(torch.bfloat16).max, -1.0  # m / root of v is 1 in the first step
    state = opt.new_state()
    opt.step([p], [g], state, step)
    flagged = infinite and param == "bf16"
    assert opt.status(state) == {"step": moe.DEV_NONFINITE_UPDATE if flagged else 0}
    assert bool(torch.isinf(p[77])) == flagged



@pytest.mark.parametrize("tensors,empty,launches", [(64, 0, 1), (64, 5, 1), (65, 0, 2), (128, 3, 2), (0, 3, 1)])
def test_launches_of_a_call(tensors, empty, launches):
    """64 tensors with elements are one launch, whatever empty ones stand around them."""
    shapes = [(0,)] * empty + [(3,)] * tensors + [(0, 2)] * empty
    opt = moe.AdamW(shapes)
    params = [torch.ones(s, device="cuda") for s in shapes]
    grads = [torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    state = opt.new_state()
    opt.step(params, grads, state, 1e-2)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(16)]
    moe.timing_attach(events)
    try:
        opt.step(params, grads, state, 1e-2)
        torch.cuda.synchronize()
        assert moe.timing_count() == launches
    finally:
        moe.timing_attach(None)
    assert state["step"].tolist() == [0, 2, 0, 0]
