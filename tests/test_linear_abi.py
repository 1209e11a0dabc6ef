"""The dense layer's entry points refuse bad arguments on the host, before anything is launched (no GPU needed)."""
import ast
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from dropless_mixture_experts_top_gb300 import _build, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = dict(T=64, K=128, N=72, act=3)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=(1 << 30) + 1), dict(T=1 << 30, K=1024), dict(K=0), dict(K=4), dict(K=100 + 1),
                                 dict(K=65544), dict(N=0), dict(N=12), dict(N=65544), dict(act=-1), dict(act=4)])
def test_configurations(L, bad):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.moe_linear_workspace(ctypes.byref(moe.LinearConfig(**GOOD)), ctypes.byref(f), ctypes.byref(b)) == 0
    assert b.value >= f.value + 64 * 72 * 2 and f.value >= 256
    assert L.moe_linear_workspace(ctypes.byref(moe.LinearConfig(**{**GOOD, **bad})), ctypes.byref(f), ctypes.byref(b)) == -1
    assert L.moe_linear_workspace(None, ctypes.byref(f), ctypes.byref(b)) == -1


# Made-up device addresses, in a child process that sees no GPU: no kernel could ever get them.
_SCRIPT = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from dropless_mixture_experts_top_gb300 import moe
L, P, B = moe.lib(), ctypes.c_void_p, ctypes.byref
res = {}
f, b = ctypes.c_size_t(), ctypes.c_size_t()
def fwd(act=3, size=0, **k):
    c = moe.LinearConfig(512, 128, 64, act)
    L.moe_linear_workspace(B(c), B(f), B(b))
    a = dict(x=0x1000, W=0x2000, bias=0x3000, residual=0x4000, y=0x5000, z=0x6000, scratch=0x7000)
    a.update(k)
    return L.moe_linear_forward(B(c), *[P(v) if v else None for v in a.values()], f.value + size, None)
def bwd(act=3, size=0, **k):
    c = moe.LinearConfig(512, 128, 64, act)
    L.moe_linear_workspace(B(c), B(f), B(b))
    a = dict(dy=0x1000, x=0x2000, W=0x3000, z=0x4000, dx=0x5000, dW=0x6000, dbias=0x7000, scratch=0x8000)
    a.update(k)
    return L.moe_linear_backward(B(c), *[P(v) if v else None for v in a.values()], b.value + size, None)
for n in ("x", "W", "y", "scratch"):
    res["fwd_null_" + n] = fwd(**{n: 0})
for n in ("x", "W", "bias", "residual", "y", "z", "scratch"):
    res["fwd_odd_" + n] = fwd(**{n: 0x9008})
res["fwd_small"] = fwd(size=-1)
res["fwd_z_without_activation"] = fwd(act=0)
for n in ("dy", "x", "W", "z", "scratch"):
    res["bwd_null_" + n] = bwd(**{n: 0})
for n in ("dy", "x", "W", "z", "dx", "dW", "dbias", "scratch"):
    res["bwd_odd_" + n] = bwd(**{n: 0x9008})
res["bwd_small"] = bwd(size=-1)
res["bwd_z_without_activation"] = bwd(act=0)
res["bwd_nothing_wanted"] = bwd(dx=0, dW=0, dbias=0)
print(repr(res))
"""


def test_refusals_before_launch(L):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    out = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    for name, rc in ast.literal_eval(out.stdout.strip().splitlines()[-1]).items():
        assert rc == (-3 if "small" in name else -2 if "odd" in name else -1), (name, rc)


def test_the_binding_s_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe._Plan, "_take_scratch", lambda self, n: torch.empty(n, dtype=torch.uint8))
    monkeypatch.setattr(moe, "_current_device", lambda: -1)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(KeyError):
        moe.Linear(4, 8, 16, activation="tanh")
    with pytest.raises(moe.MoEError):
        moe.Linear(4, 9, 16)
    lin = moe.Linear(4, 8, 16, activation="relu")
    lin._dev = -1  # where a CPU tensor says it is
    with pytest.raises(ValueError, match="bias: missing"):
        lin.forward(bf(4, 8), bf(8, 16))
    with pytest.raises(ValueError, match="W:"):
        lin.forward(bf(4, 8), bf(16, 8), bf(16))
    with pytest.raises(ValueError, match="W:"):
        lin.forward(bf(4, 8), bf(16, 8).t(), bf(16))
    with pytest.raises(ValueError, match="x:"):
        lin.forward(bf(4, 8).float(), bf(8, 16), bf(16))
    with pytest.raises(ValueError, match="dy:"):
        lin.backward(bf(4, 8), bf(4, 8), bf(8, 16), bf(4, 16))
    lin = moe.Linear(4, 8, 16, bias=False)
    lin._dev = -1
    with pytest.raises(ValueError, match="bias: given"):
        lin.forward(bf(4, 8), bf(8, 16), bf(16))



@pytest.mark.parametrize("T,K,N,fwd", [(1, 7168, 18432, 256), (2, 65536, 65536, 256), (512, 128, 64, 256), (777, 1000, 520, 256),
                                       (2048, 4096, 4096, 256), (16384, 1536, 4096, 256), (0, 64, 64, 256),
                                       (128, 30000, 64, 256 + 16 * 128 * 128 * 4), (16384, 4096, 4096, 256 + 72 * 256 * 256 * 4)])
def test_workspaces_hold_what_the_products_leave(L, T, K, N, fwd):
    """The status word; sums of the tiles that are cut into parts: none for most shapes.  The backward's: dz, and dbias' partial
    rows (four blocks on each of 152 SMs at most), and the parts of the product that has the most, a round of pairs at most."""
    for act in (0, 3):
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        assert L.moe_linear_workspace(ctypes.byref(moe.LinearConfig(T, K, N, act)), ctypes.byref(f), ctypes.byref(b)) == 0
        assert f.value == fwd
        dz = T * N * 2 if act else 0
        assert fwd + dz + N * 4 <= b.value <= 256 + 76 * 256 * 256 * 4 + dz + 608 * 64 * 4 + N * 4 + 1024
    f2, b2 = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.moe_linear_workspace(ctypes.byref(moe.LinearConfig(512, 128, 64, 0)), ctypes.byref(f2), ctypes.byref(b2)) == 0
    assert b2.value <= 256 + 8 * 64 * 4  # a small layer: no parts anywhere
