"""The gate's entry points refuse bad arguments on the host, before anything is launched (no GPU needed)."""
import ast
import ctypes
import os
import subprocess
import sys

import pytest

from dropless_mixture_experts_top_gb300 import _build, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = dict(T=64, E=32, k=4, score=0, groups=4, top_groups=2, group_best=2, renormalise=1, scale=1.0)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=(1 << 30) + 1), dict(T=1 << 29), dict(E=0), dict(E=257), dict(k=0),
                                 dict(k=17), dict(E=2, k=3), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=5),
                                 dict(groups=33, E=66), dict(top_groups=0), dict(top_groups=5), dict(group_best=0),
                                 dict(group_best=3), dict(k=9, top_groups=1), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(scale=float("nan"))])
def test_gate_configurations(L, bad):
    n = ctypes.c_size_t()
    assert L.moe_gate_workspace(ctypes.byref(moe.GateConfig(**GOOD)), ctypes.byref(n)) == 0 and n.value >= 256
    assert L.moe_gate_workspace(ctypes.byref(moe.GateConfig(**{**GOOD, **bad})), ctypes.byref(n)) == -1
    assert L.moe_gate_workspace(None, ctypes.byref(n)) == -1


# Made-up device addresses, in a child process that sees no GPU: no kernel could ever get them.
_SCRIPT = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from dropless_mixture_experts_top_gb300 import moe
L, P, B = moe.lib(), ctypes.c_void_p, ctypes.byref
res = {}
a = [P(0x100000 * (i + 1)) for i in range(12)]
odd = P(0x100008)
c = moe.GateConfig(512, 8, 2, 1, 1, 1, 1, 1, 1.0)
n = ctypes.c_size_t()
L.moe_gate_workspace(B(c), B(n))
good = [0x1000 * (i + 1) for i in range(7)]
r = moe.Routing(*good)
for i, name in enumerate(("idx", "w", "counts", "offsets", "rows", "slots", "w_row")):
    res["null_" + name] = L.moe_gate_forward(B(c), a[0], None, B(moe.Routing(*(good[:i] + [0] + good[i + 1:]))), a[1], n.value, None)
    res["odd_" + name] = L.moe_gate_forward(B(c), a[0], None, B(moe.Routing(*(good[:i] + [good[i] + 4] + good[i + 1:]))), a[1], n.value, None)
res["null_logits"] = L.moe_gate_forward(B(c), None, None, B(r), a[1], n.value, None)
res["null_routing"] = L.moe_gate_forward(B(c), a[0], None, None, a[1], n.value, None)
res["odd_bias"] = L.moe_gate_forward(B(c), a[0], odd, B(r), a[1], n.value, None)
res["null_scratch"] = L.moe_gate_forward(B(c), a[0], None, B(r), None, n.value, None)
res["small"] = L.moe_gate_forward(B(c), a[0], None, B(r), a[1], n.value - 1, None)
for i in range(5):
    args = a[:5]
    args[i] = None
    res["bwd_null_%d" % i] = L.moe_gate_backward(B(c), *args, None)
    args[i] = odd
    res["bwd_odd_%d" % i] = L.moe_gate_backward(B(c), *args, None)
res["bias_null"] = L.moe_gate_update_bias(B(c), None, a[0], 1, 0.1, None)
res["bias_null_counts"] = L.moe_gate_update_bias(B(c), a[0], None, 1, 0.1, None)
res["bias_rows"] = L.moe_gate_update_bias(B(c), a[0], a[1], -1, 0.1, None)
res["bias_odd"] = L.moe_gate_update_bias(B(c), odd, a[1], 1, 0.1, None)
print(repr(res))
"""


def test_refusals_before_launch(L):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    out = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    for name, rc in ast.literal_eval(out.stdout.strip().splitlines()[-1]).items():
        assert rc == (-3 if name == "small" else -2 if "odd" in name else -1), (name, rc)


def test_tensors_of_another_kind_are_refused(monkeypatch):
    """By the binding, with what was expected."""
    import torch
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe._Plan, "_take_scratch", lambda self, n: torch.empty(n, dtype=torch.uint8))
    monkeypatch.setattr(moe, "_current_device", lambda: None)
    g = moe.Gate(8, 4, 2)
    with pytest.raises(ValueError, match="logits|topk_idx"):
        g.forward(torch.zeros(8, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="logits"):
        g.backward(torch.zeros(4, 8).t(), *[torch.zeros(8, 2)] * 3)
    with pytest.raises(ValueError, match="bias"):
        g.update_bias(torch.zeros(5), torch.zeros(4, dtype=torch.int32), 0.1)
    with pytest.raises(KeyError):
        moe.Gate(8, 4, 2, score="tanh")
