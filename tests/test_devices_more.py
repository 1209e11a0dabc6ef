"""Plans of the gate, the dense layer and the AdamW step run on their own GPU whichever is current, and their results belong to
the stream that a call runs on (no GPU needed: stand-ins, as in test_devices.py and test_streams.py)."""
import contextlib

import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe
from tests.test_devices import OTHER, OWN, world  # noqa: F401  (a fixture)


def plans():
    z = torch.zeros
    g = moe.Gate(4, 8, 2)
    x, tk = z(4, 8), z(4, 2)
    yield g, [lambda: g.forward(x), lambda: g.forward(x, z(8)), lambda: g.backward(x, tk, tk, tk),
              lambda: g.update_bias(z(8), z(8), 0.1), g.status]
    lin = moe.Linear(4, 8, 16, activation="relu")
    lx, W, dy = z(4, 8), z(8, 16), z(4, 16)
    yield lin, [lambda: lin.forward(lx, W, z(16)), lambda: lin.backward(dy, lx, W, dy), lin.status]
    opt = moe.AdamW([(3,), (2, 2)])
    st = opt.new_state()
    ts = [z(3), z(2, 2)]
    yield opt, [lambda: opt.step(ts, ts, st, 0.1, copies=ts), lambda: opt.step(ts, ts, st, z(1), grad_scale=z(1)),
                lambda: opt.status(st)]


@pytest.mark.parametrize("current", [OWN, OTHER])
def test_a_plan_runs_on_its_own_device(world, monkeypatch, current):  # noqa: F811
    state, rec = world
    monkeypatch.setattr(moe, "_addrs", lambda ts, *a: [0] * len(ts))
    monkeypatch.setattr(moe, "_one", lambda *a: 0)
    for plan, calls in plans():
        plan._dev = OWN
        for call in calls:
            state["current"] = current
            rec.calls.clear()
            call()
            assert rec.calls and all(dev == OWN for _, dev in rec.calls), rec.calls
            assert state["current"] == current


def test_results_are_taken_on_the_call_s_stream(monkeypatch):
    taken, current = [], ["home"]

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    class Stream:
        cuda_stream = 7

        def synchronize(self):
            pass

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0
    real = torch.empty
    monkeypatch.setattr(moe, "lib", lambda: Library())
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe, "_addr", lambda *a: 0)
    monkeypatch.setattr(moe, "_current_device", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    noted = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: noted.append((t.data_ptr(), s)))
    g, lin = moe.Gate(4, 8, 2), moe.Linear(4, 8, 16, activation="relu")
    g.fwd_scratch, lin.scratch = real(512, dtype=torch.uint8), real(512, dtype=torch.uint8)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: taken.append(current[0]) or real(*a, **k))
    side = Stream()
    z = torch.zeros
    for call in (lambda s: g.forward(z(4, 8), stream=s), lambda s: g.backward(z(4, 8), z(4, 2), z(4, 2), z(4, 2), stream=s),
                 lambda s: lin.forward(z(4, 8), z(8, 16), z(16), stream=s),
                 lambda s: lin.backward(z(4, 16), z(4, 8), z(8, 16), z(4, 16), stream=s)):
        taken.clear()
        call(side)
        assert taken and all(t is side for t in taken)
        taken.clear()
        call(None)
        assert taken and all(t == "home" for t in taken)
    # the scratch is noted as in use on the other stream
    assert {p for p, s in noted} == {g.fwd_scratch.data_ptr(), lin.scratch.data_ptr()} and all(s is side for _, s in noted)
