"""The entry points around the layer refuse bad arguments on the host, before anything is launched (no GPU needed)."""
import ast
import ctypes
import os
import subprocess
import sys

import pytest

from dropless_mixture_experts_top_gb300 import _build, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=8193), dict(kind=2),
                                 dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan"))])
def test_norm_configurations(L, bad):
    good = dict(T=10, H=64, kind=0, dtype=0, eps=1e-5)
    n = ctypes.c_size_t()
    assert L.moe_norm_workspace(ctypes.byref(moe.NormConfig(**good)), ctypes.byref(n)) == 0 and n.value > 0
    assert L.moe_norm_workspace(ctypes.byref(moe.NormConfig(**{**good, **bad})), ctypes.byref(n)) == -1
    assert L.moe_norm_workspace(None, ctypes.byref(n)) == -1


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=17), dict(E=2, k=3),
                                 dict(sequences=0), dict(sequences=-1), dict(sequences=3)])
def test_balance_configurations(L, bad):
    good = dict(T=64, E=32, k=4, sequences=2)
    n = ctypes.c_size_t()
    assert L.moe_balance_workspace(ctypes.byref(moe.BalanceConfig(**good)), ctypes.byref(n)) == 0
    assert n.value >= 256
    assert L.moe_balance_workspace(ctypes.byref(moe.BalanceConfig(**{**good, **bad})), ctypes.byref(n)) == -1


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=65536), dict(R=0), dict(C=0), dict(R=16385),
                                 dict(C=16385), dict(steps=0), dict(steps=65), dict(dtype=2), dict(eps=-1.0),
                                 dict(eps=float("nan"))])
def test_ortho_configurations(L, bad):
    good = dict(batch=4, R=640, C=480, steps=5, dtype=0, eps=1e-7)
    n = ctypes.c_size_t()
    assert L.moe_ortho_workspace(ctypes.byref(moe.OrthoConfig(**good)), ctypes.byref(n)) == 0
    assert n.value >= 256 + 4 * (2 * 640 * 480 + 2 * 480 * 480) * 2
    assert L.moe_ortho_workspace(ctypes.byref(moe.OrthoConfig(**{**good, **bad})), ctypes.byref(n)) == -1


# Made-up device addresses, in a child process that sees no GPU: no kernel could ever get them.
_SCRIPT = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from dropless_mixture_experts_top_gb300 import moe
L, P, B = moe.lib(), ctypes.c_void_p, ctypes.byref
res = {}
a = [P(0x100000 * (i + 1)) for i in range(12)]
odd = P(0x100008)
c = moe.NormConfig(512, 128, 0, 0, 1e-5)
n = ctypes.c_size_t()
L.moe_norm_workspace(B(c), B(n))
res["norm_null_x"] = L.moe_norm_forward(B(c), None, None, a[1], a[2], a[3], None, a[4], None)
res["norm_sum_without_residual"] = L.moe_norm_forward(B(c), a[0], None, a[1], a[2], a[3], a[5], a[4], None)
res["norm_residual_without_sum"] = L.moe_norm_forward(B(c), a[0], a[6], a[1], a[2], a[3], None, a[4], None)
res["norm_misaligned"] = L.moe_norm_forward(B(c), odd, None, a[1], a[2], a[3], None, a[4], None)
res["norm_bwd_small"] = L.moe_norm_backward(B(c), a[0], a[1], a[2], a[3], None, a[4], a[5], a[6], a[7], n.value - 1, None)
res["norm_bwd_null_dweight"] = L.moe_norm_backward(B(c), a[0], a[1], a[2], a[3], None, a[4], None, a[6], a[7], n.value, None)
res["norm_bwd_misaligned"] = L.moe_norm_backward(B(c), a[0], a[1], a[2], a[3], odd, a[4], a[5], a[6], a[7], n.value, None)
c = moe.BalanceConfig(512, 8, 2, 1)
L.moe_balance_workspace(B(c), B(n))
res["bal_null_idx"] = L.moe_balance_forward(B(c), a[0], None, None, a[1], a[2], a[3], a[4], a[5], a[6], n.value, None)
res["bal_misaligned_mask"] = L.moe_balance_forward(B(c), a[0], a[7], odd, a[1], a[2], a[3], a[4], a[5], a[6], n.value, None)
res["bal_small"] = L.moe_balance_forward(B(c), a[0], a[7], None, a[1], a[2], a[3], a[4], a[5], a[6], n.value - 1, None)
res["bal_bwd_null"] = L.moe_balance_backward(B(c), a[0], None, a[1], a[2], 1.0, 1.0, a[3], 0, None)
res["bal_bwd_misaligned"] = L.moe_balance_backward(B(c), a[0], a[4], a[1], a[2], 1.0, 1.0, odd, 1, None)
c = moe.OrthoConfig(4, 64, 48, 1, 0, 1e-7)
L.moe_ortho_workspace(B(c), B(n))
f = (ctypes.c_float * 3)(1.5, -0.5, 0.0)
res["ortho_null_coefs"] = L.moe_ortho_update(B(c), None, a[0], None, 0.9, 1, 1.0, a[1], a[2], n.value, None)
res["ortho_null_out"] = L.moe_ortho_update(B(c), f, a[0], None, 0.9, 1, 1.0, None, a[2], n.value, None)
res["ortho_misaligned"] = L.moe_ortho_update(B(c), f, a[0], odd, 0.9, 1, 1.0, a[1], a[2], n.value, None)
res["ortho_small"] = L.moe_ortho_update(B(c), f, a[0], None, 0.9, 1, 1.0, a[1], a[2], n.value - 1, None)
print(repr(res))
"""

EXPECTED = {"norm_null_x": -1, "norm_sum_without_residual": -1, "norm_residual_without_sum": -1,
            "norm_misaligned": -2, "norm_bwd_small": -3, "norm_bwd_null_dweight": -1, "norm_bwd_misaligned": -2,
            "bal_null_idx": -1, "bal_misaligned_mask": -2, "bal_small": -3, "bal_bwd_null": -1,
            "bal_bwd_misaligned": -2, "ortho_null_coefs": -1, "ortho_null_out": -1, "ortho_misaligned": -2,
            "ortho_small": -3}


def test_refusals_before_launch(L):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    out = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    assert ast.literal_eval(out.stdout.strip().splitlines()[-1]) == EXPECTED
