"""A plan made for one GPU runs on it whichever GPU is current (no GPU needed: the library, the current device and the
tensors' addresses are stand-ins)."""
import contextlib

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe
from dropless_mixture_experts_top_gb300.synth import MoEShape

OWN, OTHER = 1, 0


class Recorder:
    """Stands in for the library: notes which device is current when an entry point is called."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.state["current"]))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    state = {"current": OWN}

    @contextlib.contextmanager
    def device(index):
        before, state["current"] = state["current"], torch.device(index).index if not isinstance(index, int) else index
        yield
        state["current"] = before

    class Stream:
        cuda_stream = 0

        def synchronize(self):
            pass
    rec = Recorder(state)
    monkeypatch.setattr(moe, "lib", lambda: rec)
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe, "_addr", lambda *a: 0)
    monkeypatch.setattr(moe, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(moe, "_current_device", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "device", device)
    return state, rec


def small(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def calls(name):
    """The calls that a plan of this kind has, on a fresh plan."""
    if name == "norm":
        n = moe.Norm(4, 8)
        x, w, st = small(4, 8), small(8), small(4, 2)
        return n, [lambda: n.forward(x, w, w), lambda: n.backward(x, x, w, st)]
    if name == "balance":
        b = moe.BalanceLoss(4, 8, 2)
        x = small(4, 8)
        return b, [lambda: b.forward(x, x), lambda: b.backward(x, x, x, x, 1.0, 1.0), b.status]
    if name == "update":
        o = moe.Orthogonaliser(1, 8, 8)
        return o, [lambda: o.update(small(1, 8, 8)), o.status]
    s = MoEShape(T=4, H=64, I=64, E=2, k=1)
    x = small(4, 64)
    if name == "router":
        r = moe.Router(s, device="cpu")
        return r, [lambda: r.forward(x, x), lambda: r.backward(x, x, x, x), r.status]
    y = moe.MoELayer(s, device="cpu")
    return y, [lambda: y.route(x), lambda: y.forward(x, x, x, x), lambda: y.recompute(x, x, x, x),
               lambda: y.backward(x, x, x, x, x), y.status]


@pytest.mark.parametrize("name", ["norm", "balance", "update", "router", "layer"])
@pytest.mark.parametrize("current", [OWN, OTHER])
def test_a_plan_runs_on_its_own_device(world, name, current):
    state, rec = world
    plan, what = calls(name)
    plan._dev = OWN
    state["current"] = current
    for call in what:
        rec.calls.clear()
        call()
        assert rec.calls and all(dev == OWN for _, dev in rec.calls), rec.calls
        assert state["current"] == current
