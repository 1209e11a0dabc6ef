"""The AdamW step refuses bad arguments on the host, before anything is launched (no GPU needed)."""
import ast
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from dropless_mixture_experts_top_gb300 import _build, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = dict(tensors=2, param_dtype=1, grad_dtype=0, state_bits=8, beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("bad", [dict(tensors=-1), dict(param_dtype=2), dict(grad_dtype=-1), dict(state_bits=16), dict(beta1=1.0),
                                 dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-9),
                                 dict(eps=float("nan")), dict(eps=float("inf"))])
def test_configurations(L, bad):
    n, out = (ctypes.c_int64 * 2)(257, 1), ctypes.c_int64()
    assert L.moe_adamw_state_elements(ctypes.byref(moe.AdamWConfig(**GOOD)), n, ctypes.byref(out)) == 0 and out.value == 768
    assert L.moe_adamw_state_elements(ctypes.byref(moe.AdamWConfig(**{**GOOD, **bad})), n, ctypes.byref(out)) == -1


@pytest.mark.parametrize("sizes", [(-1, 4), ((1 << 40) + 1, 4), (1 << 40, 1)])
def test_sizes(L, sizes):
    out = ctypes.c_int64()
    assert L.moe_adamw_state_elements(ctypes.byref(moe.AdamWConfig(**GOOD)), (ctypes.c_int64 * 2)(*sizes), ctypes.byref(out)) == -1
    assert L.moe_adamw_state_elements(ctypes.byref(moe.AdamWConfig(**GOOD)), None, ctypes.byref(out)) == -1


# Made-up device addresses, in a child process that sees no GPU: no kernel could ever get them.
_SCRIPT = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from dropless_mixture_experts_top_gb300 import moe
L, P, B = moe.lib(), ctypes.c_void_p, ctypes.byref
res = {}
good = dict(tensors=2, param_dtype=1, grad_dtype=0, state_bits=8, beta1=0.9, beta2=0.95, eps=1e-8)
ARR = P * 2
def call(c=good, n=(10, 300), decay=(0.0, 0.1), p=(0x1000, 0x2000), g=(0x3000, 0x4000), cp=(0x5000, 0), lr=0.1, lr_dev=None,
         scale=None, st=None, **state):
    s = dict(m=0x10000, v=0x20000, m_scale=0x30000, v_scale=0x40000, step=0x50000)
    s.update(state)
    st = moe.AdamWState(*[s[k] for k in ("m", "v", "m_scale", "v_scale", "step")])
    arr = lambda a: None if a is None else ARR(*a)
    return L.moe_adamw_step(B(moe.AdamWConfig(**c)), None if n is None else (ctypes.c_int64 * 2)(*n), (ctypes.c_double * 2)(*decay),
                            arr(p), arr(g), arr(cp), B(st), lr, lr_dev, scale, None)
res["config"] = call(c=dict(good, beta1=2.0))
res["sizes"] = call(n=None)
res["params"] = call(p=None)
res["grads"] = call(g=None)
res["param"] = call(p=(0x1000, 0))
res["grad"] = call(g=(0, 0x4000))
res["copies_of_bf16"] = call(c=dict(good, param_dtype=0))
res["decay"] = call(decay=(0.0, -0.1))
res["decay_nan"] = call(decay=(0.0, float("nan")))
res["lr"] = call(lr=-1.0)
res["lr_nan"] = call(lr=float("nan"))
res["odd_param"] = call(p=(0x1008, 0x2000))
res["odd_grad"] = call(g=(0x3000, 0x4004))
res["odd_copy"] = call(cp=(0x5000, 0x6002))
res["odd_lr"] = call(lr_dev=P(0x7001))
res["odd_scale"] = call(scale=P(0x7002))
for k in ("m", "v", "m_scale", "v_scale", "step"):
    res["null_" + k] = call(**{k: 0})
    res["odd_" + k] = call(**{k: 0x10008})
print(repr(res))
"""


def test_refusals_before_launch(L):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    out = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    for name, rc in ast.literal_eval(out.stdout.strip().splitlines()[-1]).items():
        assert rc == (-2 if "odd" in name else -1), (name, rc)


def test_the_binding_s_refusals(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda d: torch.device("cpu"))
    monkeypatch.setattr(moe, "_current_device", lambda: -1)
    with pytest.raises(ValueError, match="weight_decay"):
        moe.AdamW([(3,), (4,)], weight_decay=[0.1])
    with pytest.raises(ValueError, match="weight_decay"):
        moe.AdamW([(3,)], weight_decay=-0.1)
    with pytest.raises(KeyError):
        moe.AdamW([(3,)], state="4bit")
    with pytest.raises(moe.MoEError):
        moe.AdamW([(3,)], beta1=1.0)
    opt = moe.AdamW([(3,), (2, 2)])
    opt._dev = -1  # where a CPU tensor says it is
    state = opt.new_state()
    with pytest.raises(ValueError, match="params: 1 tensors"):
        opt.step([torch.zeros(3)], [torch.zeros(3)] * 2, state, 0.1)
    with pytest.raises(ValueError, match="params"):
        opt.step([torch.zeros(3), torch.zeros(4)], [torch.zeros(3)] * 2, state, 0.1)
    with pytest.raises(ValueError, match="m:"):
        opt.step([torch.zeros(3), torch.zeros(2, 2)], [torch.zeros(3)] * 2, moe.AdamW([(3,), (2, 2)], state="8bit").new_state(), 0.1)
    with pytest.raises(ValueError, match="one element"):
        moe._one(torch.zeros(2), "lr", -1)
