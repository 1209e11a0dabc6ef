"""Results that a call allocates, and a plan's scratch, belong to the stream that the call runs on (no GPU needed: the
library, the streams and the tensors' addresses are stand-ins).

The allocator hands memory out again in the order of the stream that it belongs to: a result taken from another stream's
memory may still be written by that stream's pending work, and may be handed out there while this call writes it."""
import contextlib
import ctypes
import types

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waited = handle, 0

    def synchronize(self):
        self.waited += 1


@pytest.fixture
def world(monkeypatch):
    """state: the current stream, and the stream of every allocation and every note of use so far."""
    home = Stream(1)
    state = types.SimpleNamespace(current=home, home=home, allocated=[], used=[])

    @contextlib.contextmanager
    def stream(s):
        before, state.current = state.current, s
        yield
        state.current = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                for a in args:  # sizes that are asked for
                    if isinstance(getattr(a, "_obj", None), ctypes.c_size_t):
                        a._obj.value = 512
                return 0
            return call

    def allocating(make):
        def made(*args, **kwargs):
            state.allocated.append(state.current)
            return make(*args, **kwargs)
        return made
    monkeypatch.setattr(moe, "lib", lambda: Library())
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe, "_addr", lambda *a: 0)
    monkeypatch.setattr(moe, "_current_device", lambda: None)  # the index of a plan on the CPU
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: state.current.cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state.current)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state.used.append((t.data_ptr(), s)))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, allocating(getattr(torch, f)))
    return state


def small(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def plans():
    """Each call of each plan: (a plan, its scratch, the call with a stream)."""
    n = moe.Norm(4, 8)
    x, w, st = small(4, 8), small(8), small(4, 2)
    yield "norm forward", n, None, lambda s: n.forward(x, w, w, residual=x, stream=s)
    yield "norm backward", n, n.bwd_scratch, lambda s: n.backward(x, x, w, st, stream=s)
    b = moe.BalanceLoss(4, 8, 2)
    yield "balance forward", b, b.fwd_scratch, lambda s: b.forward(x, x, stream=s)
    yield "balance backward", b, None, lambda s: b.backward(x, x, x, x, 1.0, 1.0, stream=s)
    o = moe.Orthogonaliser(1, 8, 8)
    yield "update", o, o.scratch, lambda s: o.update(small(1, 8, 8), stream=s)
    shape = MoEShape(T=4, H=64, I=64, E=2, k=1)
    y = small(4, 64)
    r = moe.Router(shape, device="cpu")
    yield "router forward", r, None, lambda s: r.forward(y, y, stream=s)
    yield "router backward", r, None, lambda s: r.backward(y, y, y, y, stream=s)
    m = moe.MoELayer(shape, device="cpu")
    yield "layer forward", m, None, lambda s: m.forward(y, y, y, y, stream=s)
    yield "layer backward", m, None, lambda s: m.backward(y, y, y, y, y, stream=s)


def test_results_belong_to_the_stream_of_the_call(world):
    other = Stream(2)
    for name, _, _, call in plans():
        for given, want in ((other, other), (None, world.home)):
            world.allocated.clear()
            call(given)
            assert world.allocated and all(s is want for s in world.allocated), name
            assert world.current is world.home


@pytest.mark.parametrize("make", [lambda: moe.Norm(4, 8), lambda: moe.BalanceLoss(4, 8, 2),
                                  lambda: moe.Orthogonaliser(1, 8, 8)])
def test_a_new_plan_is_ready_for_every_stream(world, make):
    make()
    assert world.home.waited == 1


def test_the_scratch_outlives_its_use_on_another_stream(world):
    """Dropped while another stream still works with it, it is not handed out before that work is done."""
    other = Stream(2)
    for name, plan, scratch, call in plans():
        if scratch is None:
            continue
        for at_home in (True, False):
            for given in (False, True):
                world.used.clear()
                s = world.home if at_home else other
                if given:
                    call(s)
                else:
                    with torch.cuda.stream(s):
                        call(None)
                assert world.used == ([] if at_home else [(scratch.data_ptr(), other)]), (name, at_home, given)
