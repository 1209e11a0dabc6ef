"""The gate, the dense layer and the AdamW step on a stream of their own: results that they allocate are not made in memory that
the current stream still writes, a dropped plan's scratch is not handed out while its last call runs, and calls see what
their stream did before them."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gate(kind):
    g = moe.Gate(3000, 64, 4, score="sigmoid")
    z, b, d = torch.randn(3000, 64, device="cuda"), 0.1 * torch.randn(64, device="cuda"), torch.randn(3000, 4, device="cuda")
    if kind == "forward":
        return lambda s: g.forward(z, b, stream=s)
    out = g.forward(z, b)
    return lambda s: {"d": g.backward(z, out["topk_idx"], out["topk_w"], d, stream=s)}


def linear(kind):
    lin = moe.Linear(300, 520, 264, activation="silu")
    x, W, b = (torch.randn(*s, device="cuda").to(BF) for s in ((300, 520), (520, 264), (264,)))
    dy = torch.randn(300, 264, device="cuda").to(BF)
    if kind == "forward":
        return lambda s: lin.forward(x, W, b, residual=dy, stream=s)
    return lambda s: lin.backward(dy, x, W, dy, stream=s)


@pytest.mark.parametrize("make", [gate, linear])
@pytest.mark.parametrize("kind", ["forward", "backward"])
def test_results_are_not_made_in_memory_that_is_still_written(make, kind):
    torch.manual_seed(3)
    call = make(kind)
    want = {n: t.clone() for n, t in call(None).items()}
    sizes = [(t.shape, t.dtype) for t in want.values()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    given_back = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second of the current stream
    for t in given_back:
        t.fill_(7)
    del given_back, t
    got = call(s)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("what", ["gate", "linear"])
def test_a_dropped_plan_s_scratch_is_not_handed_out_while_it_works(what):
    if what == "gate":
        plan, z = moe.Gate(60000, 256, 8), torch.randn(60000, 256, device="cuda")
        call, scratch = (lambda s: plan.forward(z, stream=s)["slot_of_row"]), plan.fwd_scratch
    else:
        plan = moe.Linear(256, 4096, 512, bias=False)
        x, W = torch.randn(256, 4096, device="cuda").to(BF), torch.randn(4096, 512, device="cuda").to(BF)
        call, scratch = (lambda s: plan.forward(x, W, stream=s)["y"]), plan.scratch
    want, size, at = call(None).clone(), scratch.numel(), scratch.data_ptr()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    got = call(s)
    del plan, call, scratch
    taken = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert taken.data_ptr() != at
    taken.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_steps_in_the_order_of_their_stream():
    opt = moe.AdamW([(5000,), (33, 7)], state="8bit", beta2=0.95)
    params = [torch.randn(s, device="cuda") for s in ((5000,), (33, 7))]
    twin, st, tst = [p.clone() for p in params], opt.new_state(), opt.new_state()
    grads = [torch.zeros(s, device="cuda", dtype=BF) for s in ((5000,), (33, 7))]
    new = [[torch.randn(g.shape, device="cuda").to(BF) for g in grads] for _ in range(3)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for g3 in new:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            for g, v in zip(grads, g3):
                g.copy_(v)
        opt.step(params, grads, st, 0.01, stream=s)
    torch.cuda.synchronize()
    for g3 in new:
        opt.step(twin, g3, tst, 0.01)
    assert all(torch.equal(a, b) for a, b in zip(params, twin))
    assert opt.status(st, s) == {"step": 0}


def test_long_tensors():
    """Past 2^31 elements: offsets of rows and of single elements."""
    T, E = 8_500_000, 256
    z = torch.zeros(T, E, device="cuda")
    z[:, 200] = 1.0
    z[-1000:] = torch.randn(1000, E, device="cuda")
    g = moe.Gate(T, E, 1, score="sigmoid", renormalise=False)
    out = g.forward(z)
    assert torch.equal(out["topk_idx"][-1000:, 0].long(), z[-1000:].argmax(1))
    assert int(out["counts"].sum()) == T and int(out["counts"][200]) >= T - 1000
    torch.testing.assert_close(out["topk_w"][-1000:, 0], torch.sigmoid(z[-1000:].max(1).values))
    d = g.backward(z, out["topk_idx"], out["topk_w"], torch.ones(T, 1, device="cuda"))
    w = out["topk_w"][-1000:, 0]
    torch.testing.assert_close(d[-1000:].sum(1), w * (1 - w), rtol=1e-5, atol=1e-7)
    del z, d, out
    T, K, N = 600_000, 64, 4096
    x, W = torch.randint(-2, 3, (T, K), device="cuda").to(BF), torch.randint(-2, 3, (K, N), device="cuda").to(BF)
    lin = moe.Linear(T, K, N, activation="relu", bias=False)
    out = lin.forward(x, W)
    for rows in (slice(0, 100), slice(524_200, 524_400), slice(T - 100, T)):
        ref = (x[rows].double() @ W.double())
        assert torch.equal(out["z"][rows], ref.to(BF)) and torch.equal(out["y"][rows], ref.clamp(min=0).to(BF))
    got = lin.backward(out["y"], x, W, out["z"])
    for rows in (slice(0, 100), slice(T - 100, T)):
        dz = out["y"][rows].double()
        ref = dz @ W.double().T  # (sums below 2^24: exact)
        assert torch.equal(got["dx"][rows], ref.to(BF))
