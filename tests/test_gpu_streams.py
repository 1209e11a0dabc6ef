"""Calls on a stream of their own, with results that they allocate, while the current stream still writes memory that it
has given back: none of that memory may be what the results are made in."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


def norm(kind):
    n = moe.Norm(256, 512)
    x, r = (torch.randn(256, 512, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(512, device="cuda").to(torch.bfloat16)
    st = torch.rand(256, 2, device="cuda")
    if kind == "forward":
        return lambda s: n.forward(x, w, w, residual=r, stream=s)
    return lambda s: n.backward(x, r, w, st, d_sum=r, stream=s)


def balance(kind):
    b = moe.BalanceLoss(4096, 64, 2, sequences=4)
    lg = torch.randn(4096, 64, device="cuda")
    idx = torch.topk(lg, 2, dim=1).indices.to(torch.int32)
    if kind == "forward":
        return lambda s: b.forward(lg, idx, stream=s)
    out = b.forward(lg, idx)
    return lambda s: {"d": b.backward(lg, out["counts"], out["tokens"], out["lse"], 1.0, 0.1, stream=s)}


def update(kind):
    o = moe.Orthogonaliser(3, 200, 304)
    g = torch.randn(3, 200, 304, device="cuda").to(torch.bfloat16)
    return lambda s: {"out": o.update(g, stream=s)}


def router(kind):
    r = moe.Router(MoEShape(T=256, H=128, I=64, E=16, k=2))
    x = torch.randn(256, 128, device="cuda").to(torch.bfloat16).view(torch.int16)
    w = torch.randn(128, 16, device="cuda").to(torch.bfloat16).view(torch.int16)
    return lambda s: {"logits": r.forward(x, w, stream=s)}


@pytest.mark.parametrize("make,kind", [(norm, "forward"), (norm, "backward"), (balance, "forward"),
                                       (balance, "backward"), (update, ""), (router, "")])
def test_results_are_not_made_in_memory_that_is_still_written(make, kind):
    torch.manual_seed(3)
    call = make(kind)
    want = {n: t.clone() for n, t in call(None).items() if t is not None}
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


def test_a_dropped_plan_s_scratch_is_not_handed_out_while_it_works():
    g = torch.randn(6, 1024, 1024, device="cuda").to(torch.bfloat16)
    o = moe.Orthogonaliser(6, 1024, 1024)
    want = o.update(g)
    size = o.scratch.numel()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    got = o.update(g, stream=s)
    at = o.scratch.data_ptr()
    del o
    taken = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert taken.data_ptr() != at
    taken.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
