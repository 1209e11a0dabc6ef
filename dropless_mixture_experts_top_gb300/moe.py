"""Thin ctypes binding of libmoe_gb300.so (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  There is no fallback:
if the library is missing or the GPU is not an sm_103a part, calls raise.

Low-level functions mirror the C names (query_workspace, route, forward,
backward, get_device_status, status_string, timing_*).  `MoELayer` bundles the
buffers one configuration needs.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

from . import _build

MOE_OK = 0
PRECISIONS = {"bf16": 0, "fp8_bwd": 1, "mxfp8": 2}
DEV_NONFINITE_LOGIT = 0x1
DEV_WAIT_TIMEOUT = 0x2
DEV_NONFINITE_UPDATE = 0x4
DEV_BAD_INDEX = 0x8

_lib = None

EXPORTED = [
    "moe_query_workspace", "moe_saved_offsets", "moe_fp8_scratch_offsets", "moe_mxfp8_forward_offsets",
    "moe_route",
    "moe_route_static_scratch", "moe_forward", "moe_forward_nosave", "moe_forward_recompute", "moe_backward",
    "moe_get_device_status",
    "moe_status_string", "moe_timing_attach", "moe_timing_count", "moe_timing_label",
    "moe_selftest_wait_timeout", "moe_router_workspace", "moe_router_forward", "moe_router_backward",
    "moe_norm_workspace", "moe_norm_forward", "moe_norm_backward",
    "moe_balance_workspace", "moe_balance_forward", "moe_balance_backward",
    "moe_ortho_workspace", "moe_ortho_update",
]


class Config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("precision", ctypes.c_int32)]


class Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "counts", "offsets", "row_of_slot", "slot_of_row", "w_row")]


class NormConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class BalanceConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "k", "sequences")]


class OrthoConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "R", "C", "steps", "dtype")] + [("eps", ctypes.c_float)]


class SavedLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("x_perm", "G", "U", "A", "Y", "A_w")]


class Fp8Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "m_pad", "pad_offsets", "dy_q", "dy_sf", "wd_q", "wd_sf", "dg_q", "dg_sf", "du_q", "du_sf",
        "wg_q", "wg_sf", "wu_q", "wu_sf", "aw_t", "aw_t_sf", "dy_t", "dy_t_sf", "x_t", "x_t_sf",
        "dg_t", "dg_t_sf", "du_t", "du_t_sf")]


class Mx8FwdLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "m_pad", "pad_offsets", "x_q", "x_sf", "a_q", "a_sf", "wgu_q", "wgu_sf", "wdt_q", "wdt_sf",
        "bwd_wd_q", "bwd_wd_sf", "bwd_wg_q", "bwd_wg_sf", "bwd_wu_q", "bwd_wu_sf")]


class MoEError(RuntimeError):
    def __init__(self, what, code):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def lib():
    """Load the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(path)
        P, sz = ctypes.c_void_p, ctypes.c_size_t
        L.moe_query_workspace.argtypes = [P, P, P, P, P]
        L.moe_saved_offsets.argtypes = [P, P]
        L.moe_fp8_scratch_offsets.argtypes = [P, P]
        L.moe_mxfp8_forward_offsets.argtypes = [P, P]
        L.moe_route.argtypes = [P, P, P, P, sz, P]
        L.moe_forward.argtypes = [P, P, P, P, P, P, P, P, sz, P, sz, P]
        L.moe_forward_nosave.argtypes = [P, P, P, P, P, P, P, P, sz, P, sz, P]
        L.moe_forward_recompute.argtypes = [P, P, P, P, P, P, P, sz, P, sz, P]
        L.moe_backward.argtypes = [P, P, P, P, P, P, P, P, sz, P, P, P, P, P, P, P, sz, P]
        L.moe_get_device_status.argtypes = [P, P, P]
        L.moe_selftest_wait_timeout.argtypes = [P, P]
        L.moe_selftest_wait_timeout.restype = ctypes.c_int
        L.moe_router_workspace.argtypes = [P, P, P]
        L.moe_router_forward.argtypes = [P, P, P, P, P, sz, P]
        L.moe_router_backward.argtypes = [P, P, P, P, P, P, P, sz, P]
        for f in ("moe_router_workspace", "moe_router_forward", "moe_router_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.moe_norm_workspace.argtypes = [P, P]
        L.moe_norm_forward.argtypes = [P] * 9
        L.moe_norm_backward.argtypes = [P] * 10 + [sz, P]
        L.moe_balance_workspace.argtypes = [P, P]
        L.moe_balance_forward.argtypes = [P] * 10 + [sz, P]
        L.moe_balance_backward.argtypes = [P] * 5 + [ctypes.c_float, ctypes.c_float, P, ctypes.c_int32, P]
        L.moe_ortho_workspace.argtypes = [P, P]
        L.moe_ortho_update.argtypes = [P, P, P, P, ctypes.c_float, ctypes.c_int32, ctypes.c_float, P, P, sz, P]
        for f in ("moe_ortho_workspace", "moe_ortho_update", "moe_norm_workspace", "moe_norm_forward", "moe_norm_backward", "moe_balance_workspace",
                  "moe_balance_forward", "moe_balance_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_timing_attach.argtypes = [P, ctypes.c_int32]
        L.moe_timing_count.argtypes = []
        L.moe_timing_count.restype = ctypes.c_int32
        L.moe_timing_label.argtypes = [ctypes.c_int32]
        L.moe_timing_label.restype = ctypes.c_char_p
        for f in ("moe_query_workspace", "moe_saved_offsets", "moe_fp8_scratch_offsets",
                  "moe_mxfp8_forward_offsets", "moe_route", "moe_forward", "moe_backward",
                  "moe_get_device_status", "moe_timing_attach"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def _check(code, what):
    if code != MOE_OK:
        raise MoEError(what, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_config(shape, precision="bf16") -> Config:
    return Config(int(shape.T), int(shape.H), int(shape.I), int(shape.E), int(shape.k),
                  PRECISIONS[precision] if isinstance(precision, str) else int(precision))


def query_workspace(cfg: Config):
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().moe_query_workspace(ctypes.byref(cfg), *[ctypes.byref(o) for o in out]),
           "moe_query_workspace")
    return tuple(int(o.value) for o in out)


def saved_offsets(cfg: Config) -> dict:
    lay = SavedLayout()
    _check(lib().moe_saved_offsets(ctypes.byref(cfg), ctypes.byref(lay)), "moe_saved_offsets")
    return {n: int(getattr(lay, n)) for n, _ in SavedLayout._fields_}


def fp8_scratch_offsets(cfg: Config) -> dict:
    lay = Fp8Layout()
    _check(lib().moe_fp8_scratch_offsets(ctypes.byref(cfg), ctypes.byref(lay)),
           "moe_fp8_scratch_offsets")
    return {n: int(getattr(lay, n)) for n, _ in Fp8Layout._fields_}


def mxfp8_forward_offsets(cfg: Config) -> dict:
    lay = Mx8FwdLayout()
    _check(lib().moe_mxfp8_forward_offsets(ctypes.byref(cfg), ctypes.byref(lay)),
           "moe_mxfp8_forward_offsets")
    return {n: int(getattr(lay, n)) for n, _ in Mx8FwdLayout._fields_}


MX_BN = 192  # N extent of an MXFP8 GEMM tile: B-operand scales are grouped by it


def sf_grouping(base: str, shape, m_pad: int):
    """(segment rows, group rows) of a quantised operand's scale atoms."""
    if base in ("wd_q",):
        return shape.I, MX_BN
    if base in ("wg_q", "wu_q"):
        return shape.H, MX_BN
    if base == "dy_t":
        return shape.H, MX_BN
    if base in ("dg_t", "du_t"):
        return shape.I, MX_BN
    if base == "wgu_q":
        return 2 * shape.I, MX_BN
    if base == "wdt_q":
        return shape.H, MX_BN
    rows = {"dy_q": m_pad, "dg_q": m_pad, "du_q": m_pad, "aw_t": shape.I, "x_t": shape.H,
            "x_q": m_pad, "a_q": m_pad}[base]
    return rows, 128


def sf_layout_bytes(rows: int, K: int, seg: int, group: int) -> int:
    nseg, gps, apg = -(-rows // seg), -(-seg // group), -(-group // 128)
    return nseg * gps * apg * (K // 128) * 512


def make_routing(r: dict) -> Routing:
    return Routing(*[r[n].data_ptr() for n, _ in Routing._fields_])


def route(cfg, logits, routing: dict, scratch, stream=None):
    rt = make_routing(routing)
    _check(lib().moe_route(ctypes.byref(cfg), _ptr(logits), ctypes.byref(rt), _ptr(scratch),
                           scratch.numel(), _stream(stream)), "moe_route")


def forward(cfg, x, routing: dict, W_gate, W_up, W_down, out, saved, scratch, stream=None, save=True):
    """moe_forward, or moe_forward_nosave when save is False (out only)."""
    rt = make_routing(routing)
    fn, name = (lib().moe_forward, "moe_forward") if save else (lib().moe_forward_nosave, "moe_forward_nosave")
    _check(fn(ctypes.byref(cfg), _ptr(x), ctypes.byref(rt), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(out),
              _ptr(saved), saved.numel(), _ptr(scratch), scratch.numel(), _stream(stream)), name)


def forward_recompute(cfg, x, routing: dict, W_gate, W_up, W_down, saved, scratch, stream=None):
    rt = make_routing(routing)
    _check(lib().moe_forward_recompute(ctypes.byref(cfg), _ptr(x), ctypes.byref(rt), _ptr(W_gate), _ptr(W_up),
                                       _ptr(W_down), _ptr(saved), saved.numel(), _ptr(scratch), scratch.numel(),
                                       _stream(stream)), "moe_forward_recompute")


def backward(cfg, dy, x, routing: dict, W_gate, W_up, W_down, saved, dx, dW_gate, dW_up, dW_down,
             d_logits, d_topk_w, scratch, stream=None):
    rt = make_routing(routing)
    _check(lib().moe_backward(ctypes.byref(cfg), _ptr(dy), _ptr(x), ctypes.byref(rt), _ptr(W_gate),
                              _ptr(W_up), _ptr(W_down), _ptr(saved), saved.numel(), _ptr(dx),
                              _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), _ptr(d_logits),
                              _ptr(d_topk_w), _ptr(scratch), scratch.numel(), _stream(stream)),
           "moe_backward")


def get_device_status(scratch, stream=None) -> int:
    code = ctypes.c_int32()
    rc = lib().moe_get_device_status(_ptr(scratch), _stream(stream), ctypes.byref(code))
    if rc not in (MOE_OK, -6):
        _check(rc, "moe_get_device_status")
    return int(code.value)


def router_workspace(cfg: Config):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_router_workspace(ctypes.byref(cfg), ctypes.byref(f), ctypes.byref(b)),
           "moe_router_workspace")
    return int(f.value), int(b.value)


def _device(device):
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"device: {d}, expected a GPU")
    return torch.device("cuda", torch.cuda.current_device()) if d.index is None else d


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # (without its Python layers)


def _on_own_device(call):
    """A plan's method, run with the plan's GPU current: the library launches on the current one.  The three plans
    whose smallest calls are a few microseconds ask for themselves: this wrapper costs 0.4 of one."""
    @functools.wraps(call)
    def on_own_device(self, *args, **kwargs):
        if _current_device() == self._dev:
            return call(self, *args, **kwargs)
        with torch.cuda.device(self._dev):
            return call(self, *args, **kwargs)
    return on_own_device


def _on_stream(stream):
    """Where the results of a call on this stream (None: the current one) are allocated: memory is handed out again in
    the order of the stream that it was taken on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class Router:
    """The router projection logits = x . W_r (bf16 in, fp32 logits) and its
    backward, over scratch buffers sized for one configuration."""

    def __init__(self, shape, device="cuda"):
        self.shape = shape
        self.cfg = make_config(shape)
        fs, bs = router_workspace(self.cfg)
        self.fwd_scratch = torch.empty(fs, dtype=torch.uint8, device=device)
        self.bwd_scratch = torch.empty(bs, dtype=torch.uint8, device=device)
        self.device, self._dev = device, _device(device).index

    @_on_own_device
    def forward(self, x, W_r, logits=None, stream=None):
        if logits is None:
            with _on_stream(stream):
                logits = torch.empty((self.shape.T, self.shape.E), dtype=torch.float32, device=self.device)
        _check(lib().moe_router_forward(ctypes.byref(self.cfg), _ptr(x), _ptr(W_r), _ptr(logits),
                                        _ptr(self.fwd_scratch), self.fwd_scratch.numel(), _stream(stream)),
               "moe_router_forward")
        return logits

    @_on_own_device
    def backward(self, x, W_r, d_logits, dx, dW_r=None, stream=None):
        """dx (bf16 [T,H]) is updated in place; returns dW_r (fp32 [H,E])."""
        if dW_r is None:
            with _on_stream(stream):
                dW_r = torch.empty((self.shape.H, self.shape.E), dtype=torch.float32, device=self.device)
        _check(lib().moe_router_backward(ctypes.byref(self.cfg), _ptr(x), _ptr(W_r), _ptr(d_logits), _ptr(dx),
                                         _ptr(dW_r), _ptr(self.bwd_scratch), self.bwd_scratch.numel(),
                                         _stream(stream)), "moe_router_backward")
        return dW_r

    @_on_own_device
    def status(self, stream=None) -> dict:
        return {n: get_device_status(b, stream) for n, b in (("forward", self.fwd_scratch),
                                                             ("backward", self.bwd_scratch))}


# ---- around the layer: the norm, the balance loss and the orthogonalised update

DTYPES = {"bf16": 0, "fp32": 1}
NORM_KINDS = {"layer": 0, "rms": 1}
# what a tensor of each type may be: bf16 also as the int16 view of its bits
_BF16 = (torch.bfloat16, torch.int16)
_TORCH_DTYPES = {"bf16": _BF16, "fp32": (torch.float32,)}


def _addr(t, name, shape, dtypes, dev):
    """The address of a tensor argument (None: no address), which has to be a dense
    tensor of this shape and one of these types on GPU dev."""
    if t is None:
        return None
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, {'' if t.is_contiguous() else 'not '}"
                     f"contiguous; expected one of {dtypes}, {tuple(shape)}, on GPU {dev}, contiguous")


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


class _Plan:
    """A plan's scratch and the streams that work with it."""

    def _take_scratch(self, n):
        """A scratch buffer whose status reads 0 before its first call, ready for use on any stream."""
        s = torch.empty(n, dtype=torch.uint8, device=self.device)
        s[:256] = 0
        torch.cuda.current_stream(self.device).synchronize()
        self._home = _raw_stream(None, self._dev)
        return s

    def _working(self, scratch, stream):
        """The handle of the stream that a call works on.  The allocator is told where that is not the stream that the
        scratch was taken on: a plan may be dropped while its last call runs."""
        raw = _raw_stream(stream, self._dev)
        if raw != self._home:
            scratch.record_stream(torch.cuda.current_stream(self._dev) if stream is None else stream)
        return raw


class Norm(_Plan):
    """Layer norm (kind "layer") or RMS norm ("rms") over [T, H] of one type
    ("bf16" or "fp32"), with the residual sum in front of it, and its backward.

    Dictionaries that a call returned may be handed to the next one, which then
    writes into the same tensors.  Outputs have the type of x (or dy); the
    statistics and the weight's gradients are fp32."""

    def __init__(self, T, H, kind="layer", dtype="bf16", bias=True, eps=1e-5, device="cuda"):
        self.cfg = NormConfig(int(T), int(H), NORM_KINDS[kind], DTYPES[dtype], float(eps))
        n = ctypes.c_size_t()
        _check(lib().moe_norm_workspace(ctypes.byref(self.cfg), ctypes.byref(n)), "moe_norm_workspace")
        self.device, self.bias = _device(device), bool(bias)
        self._dev, self._fwd, self._bwd = self.device.index, lib().moe_norm_forward, lib().moe_norm_backward
        self._cfg, self._types = ctypes.byref(self.cfg), _TORCH_DTYPES[dtype]
        self._rows, self._cols, self._stats = (torch.Size(s) for s in ((T, H), (H,), (T, 2)))
        self.bwd_scratch = self._take_scratch(n.value)
        self._scratch = self.bwd_scratch.data_ptr()

    def forward(self, x, weight, bias=None, residual=None, out=None, stream=None) -> dict:
        """{"y", "sum" (x + residual, or None), "stats" [T, 2]: mean and 1 / deviation}"""
        d, ty, rows, cols = self._dev, self._types, self._rows, self._cols
        if _current_device() != d:
            with torch.cuda.device(d):
                return self.forward(x, weight, bias, residual, out, stream)
        if (bias is not None) != self.bias:
            raise ValueError("bias: given to a norm without one" if bias is not None else "bias: missing")
        if out is None:
            with _on_stream(stream):
                out = {"y": torch.empty_like(x), "sum": torch.empty_like(x) if residual is not None else None,
                       "stats": torch.empty(self._stats, dtype=torch.float32, device=self.device)}
        rc = self._fwd(
            self._cfg, _addr(x, "x", rows, ty, d), _addr(residual, "residual", rows, ty, d),
            _addr(weight, "weight", cols, ty, d), _addr(bias, "bias", cols, ty, d), _addr(out["y"], "y", rows, ty, d),
            _addr(out["sum"], "sum", rows, ty, d), _addr(out["stats"], "stats", self._stats, _F32, d),
            _raw_stream(stream, d))
        if rc:
            raise MoEError("moe_norm_forward", rc)
        return out

    def backward(self, dy, h, weight, stats, d_sum=None, grads=None, stream=None) -> dict:
        """{"dx", "dweight", "dbias" (None without a bias)} from the forward's
        stats and h, its sum (x where there was no residual)."""
        d, ty, rows, cols = self._dev, self._types, self._rows, self._cols
        if _current_device() != d:
            with torch.cuda.device(d):
                return self.backward(dy, h, weight, stats, d_sum, grads, stream)
        if grads is None:
            f32 = dict(dtype=torch.float32, device=self.device)
            with _on_stream(stream):
                grads = {"dx": torch.empty_like(dy), "dweight": torch.empty(cols, **f32),
                         "dbias": torch.empty(cols, **f32) if self.bias else None}
        rc = self._bwd(
            self._cfg, _addr(dy, "dy", rows, ty, d), _addr(h, "h", rows, ty, d),
            _addr(weight, "weight", cols, ty, d), _addr(stats, "stats", self._stats, _F32, d),
            _addr(d_sum, "d_sum", rows, ty, d), _addr(grads["dx"], "dx", rows, ty, d),
            _addr(grads["dweight"], "dweight", cols, _F32, d), _addr(grads["dbias"], "dbias", cols, _F32, d),
            self._scratch, self.bwd_scratch.numel(), self._working(self.bwd_scratch, stream))
        if rc:
            raise MoEError("moe_norm_backward", rc)
        return grads


_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8, torch.bool)


class BalanceLoss(_Plan):
    """The router's balance loss and z loss over `sequences` equal parts of T
    tokens, with per-expert counts, and their gradient for the logits."""

    def __init__(self, T, E, k, sequences=1, device="cuda"):
        self.cfg = BalanceConfig(int(T), int(E), int(k), int(sequences))
        n = ctypes.c_size_t()
        _check(lib().moe_balance_workspace(ctypes.byref(self.cfg), ctypes.byref(n)), "moe_balance_workspace")
        self.device, self._cfg = _device(device), ctypes.byref(self.cfg)
        self._dev, self._fwd, self._bwd = self.device.index, lib().moe_balance_forward, lib().moe_balance_backward
        self._te, self._tk, self._t, self._se, self._s, self._two = (
            torch.Size(s) for s in ((T, E), (T, k), (T,), (sequences, E), (sequences,), (2,)))
        self.fwd_scratch = self._take_scratch(n.value)
        self._scratch = self.fwd_scratch.data_ptr()

    def forward(self, logits, topk_idx, mask=None, out=None, stream=None) -> dict:
        """{"loss" [2]: balance, z; "counts" and "probs" [sequences, E]; "tokens"
        [sequences]; "lse" [T]}.  mask [T]: zero for padding."""
        d = self._dev
        if _current_device() != d:
            with torch.cuda.device(d):
                return self.forward(logits, topk_idx, mask, out, stream)
        if out is None:
            f32, i32 = (dict(dtype=t, device=self.device) for t in (torch.float32, torch.int32))
            with _on_stream(stream):
                out = {"loss": torch.empty(self._two, **f32), "counts": torch.empty(self._se, **i32),
                       "probs": torch.empty(self._se, **f32), "tokens": torch.empty(self._s, **i32),
                       "lse": torch.empty(self._t, **f32)}
        rc = self._fwd(
            self._cfg, _addr(logits, "logits", self._te, _F32, d), _addr(topk_idx, "topk_idx", self._tk, _I32, d),
            _addr(mask, "mask", self._t, _U8, d), _addr(out["loss"], "loss", self._two, _F32, d),
            _addr(out["counts"], "counts", self._se, _I32, d), _addr(out["probs"], "probs", self._se, _F32, d),
            _addr(out["tokens"], "tokens", self._s, _I32, d), _addr(out["lse"], "lse", self._t, _F32, d),
            self._scratch, self.fwd_scratch.numel(), self._working(self.fwd_scratch, stream))
        if rc:
            raise MoEError("moe_balance_forward", rc)
        return out

    def backward(self, logits, counts, tokens, lse, g_balance, g_z, d_logits=None, stream=None):
        """The gradient of g_balance * loss[0] + g_z * loss[1], added to d_logits in
        place where that is given (as the layer's backward left it)."""
        d, add = self._dev, d_logits is not None
        if _current_device() != d:
            with torch.cuda.device(d):
                return self.backward(logits, counts, tokens, lse, g_balance, g_z, d_logits, stream)
        if not add:
            with _on_stream(stream):
                d_logits = torch.empty(self._te, dtype=torch.float32, device=self.device)
        rc = self._bwd(
            self._cfg, _addr(logits, "logits", self._te, _F32, d), _addr(counts, "counts", self._se, _I32, d),
            _addr(tokens, "tokens", self._s, _I32, d), _addr(lse, "lse", self._t, _F32, d), g_balance, g_z,
            _addr(d_logits, "d_logits", self._te, _F32, d), add, _raw_stream(stream, d))
        if rc:
            raise MoEError("moe_balance_backward", rc)
        return d_logits

    @_on_own_device
    def status(self, stream=None) -> dict:
        return {"forward": get_device_status(self.fwd_scratch, stream)}


# the quintic Newton-Schulz step whose five-fold use is the Muon optimiser's
MUON_COEFS = ((3.4445, -4.7750, 2.0315),) * 5


class Orthogonaliser(_Plan):
    """The orthogonalised update of `batch` matrices [R, C] by Newton-Schulz
    products, optionally through a momentum, over a scratch buffer of its own.
    coefs: one (a, b, c) per step."""

    def __init__(self, batch, R, C, dtype="bf16", coefs=MUON_COEFS, eps=1e-7, device="cuda"):
        coefs = [float(v) for step in coefs for v in step]
        if not coefs or len(coefs) % 3:
            raise ValueError("coefs: three numbers for each of one or more steps")
        self.cfg = OrthoConfig(int(batch), int(R), int(C), len(coefs) // 3, DTYPES[dtype], float(eps))
        n = ctypes.c_size_t()
        _check(lib().moe_ortho_workspace(ctypes.byref(self.cfg), ctypes.byref(n)), "moe_ortho_workspace")
        self.device, self._cfg, self._types = _device(device), ctypes.byref(self.cfg), _TORCH_DTYPES[dtype]
        self._shape = torch.Size((batch, R, C))
        self._dev, self._update = self.device.index, lib().moe_ortho_update
        self._coefs = (ctypes.c_float * len(coefs))(*coefs)
        self.scratch = self._take_scratch(n.value)
        self._scratch = self.scratch.data_ptr()

    def update(self, g, momentum=None, beta=0.95, nesterov=True, scale=1.0, out=None, stream=None):
        """scale times the orthogonalised update, bf16 [batch, R, C]; momentum (fp32)
        is advanced in place."""
        d, s = self._dev, self._shape
        if _current_device() != d:
            with torch.cuda.device(d):
                return self.update(g, momentum, beta, nesterov, scale, out, stream)
        if out is None:
            with _on_stream(stream):
                out = torch.empty(s, dtype=g.dtype if g.dtype in _BF16 else torch.bfloat16, device=self.device)
        rc = self._update(
            self._cfg, self._coefs, _addr(g, "g", s, self._types, d), _addr(momentum, "momentum", s, _F32, d), beta,
            nesterov, scale, _addr(out, "out", s, _BF16, d), self._scratch, self.scratch.numel(),
            self._working(self.scratch, stream))
        if rc:
            raise MoEError("moe_ortho_update", rc)
        return out

    @_on_own_device
    def status(self, stream=None) -> dict:
        return {"update": get_device_status(self.scratch, stream)}


def selftest_wait_timeout(status, stream=None):
    """Launch the bounded-wait diagnostic; `status` is a device int32 tensor."""
    _check(lib().moe_selftest_wait_timeout(_ptr(status), _stream(stream)), "moe_selftest_wait_timeout")


def timing_attach(events):
    """events: list of torch.cuda.Event (enable_timing=True), two per kernel.
    torch creates the CUDA event object lazily, so each one is recorded once here
    to make its handle valid."""
    global _timing_keep
    if events is None:
        _check(lib().moe_timing_attach(None, 0), "moe_timing_attach")
        _timing_keep = None
        return
    for e in events:
        e.record()
    torch.cuda.synchronize()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _timing_keep = arr
    _check(lib().moe_timing_attach(arr, len(events) // 2), "moe_timing_attach")


_timing_keep = None


def timing_count() -> int:
    return int(lib().moe_timing_count())


def timing_label(i: int) -> str:
    s = lib().moe_timing_label(int(i))
    return s.decode() if s else ""


def bf16_view(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.bfloat16)


class MoELayer:
    """Device buffers for one configuration, and the three calls over them."""

    def __init__(self, shape, precision="bf16", device="cuda"):
        self.shape = shape
        self.cfg = make_config(shape, precision)
        self.device, self._dev = torch.device(device), _device(device).index
        T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
        rs, sv, fs, bs = query_workspace(self.cfg)
        dev = self.device
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.routing = {
            "topk_idx": torch.empty((T, k), dtype=i32, device=dev),
            "topk_w": torch.empty((T, k), dtype=f32, device=dev),
            "counts": torch.empty((E,), dtype=i32, device=dev),
            "offsets": torch.empty((E + 1,), dtype=i32, device=dev),
            "row_of_slot": torch.empty((T, k), dtype=i32, device=dev),
            "slot_of_row": torch.empty((T * k,), dtype=i32, device=dev),
            "w_row": torch.empty((T * k,), dtype=f32, device=dev),
        }
        self.route_scratch = torch.empty(rs, dtype=u8, device=dev)
        self.saved = torch.empty(sv, dtype=u8, device=dev)
        self.fwd_scratch = torch.empty(fs, dtype=u8, device=dev)
        self.bwd_scratch = torch.empty(bs, dtype=u8, device=dev)
        self.saved_offsets = saved_offsets(self.cfg)

    def saved_tensor(self, name):
        T, H, I, k = self.shape.T, self.shape.H, self.shape.I, self.shape.k
        cols = H if name in ("x_perm", "Y") else I
        off = self.saved_offsets[name]
        n = T * k * cols
        return self.saved[off:off + 2 * n].view(torch.int16).view(T * k, cols)

    def fp8_tensor(self, name):
        """A quantised operand left in the backward scratch (the fp8 modes), or for
        aw_t (w * A along tokens), x_t (x along tokens) and the weights' wd_q, wg_q,
        wu_q (all written by the forward) in `saved`: uint8 codes [rows, K] for *_q and *_t, the raw
        scale-atom bytes for *_sf, int32 [E+1] for pad_offsets."""
        lay = fp8_scratch_offsets(self.cfg)
        s = self.shape
        Mp = lay["m_pad"]
        rows_k = {"dy_q": (Mp, s.H), "wd_q": (s.E * s.I, s.H), "dg_q": (Mp, s.I), "du_q": (Mp, s.I),
                  "wg_q": (s.E * s.H, s.I), "wu_q": (s.E * s.H, s.I), "aw_t": (s.I, Mp),
                  "dy_t": (s.H, Mp), "x_t": (s.H, Mp), "dg_t": (s.I, Mp), "du_t": (s.I, Mp)}
        off = lay[name]
        in_saved = name.startswith(("aw_t", "x_t", "wd_", "wg_", "wu_"))  # written by the forward
        buf = self.saved if in_saved else self.bwd_scratch
        if name == "pad_offsets":
            return buf[off:off + 4 * (s.E + 1)].view(torch.int32)
        if name.endswith("_sf"):
            base = name[:-3] + "_q" if name[:-3] + "_q" in rows_k else name[:-3]
            R, K = rows_k[base]
            seg, group = sf_grouping(base, s, Mp)
            return buf[off:off + sf_layout_bytes(R, K, seg, group)]
        R, K = rows_k[name]
        return buf[off:off + R * K].view(R, K)

    def fwd_fp8_tensor(self, name):
        """A quantised operand of the mxfp8 forward: in the forward scratch, or for
        bwd_* (the backward's weight operands) in `saved`.  uint8 codes [rows, K]
        for *_q, raw scale-atom bytes for *_sf, int32 [E+1] for pad_offsets."""
        lay = mxfp8_forward_offsets(self.cfg)
        s = self.shape
        Mp = lay["m_pad"]
        rows_k = {"x_q": (Mp, s.H), "a_q": (Mp, s.I), "wgu_q": (s.E * 2 * s.I, s.H), "wdt_q": (s.E * s.H, s.I),
                  "bwd_wd_q": (s.E * s.I, s.H), "bwd_wg_q": (s.E * s.H, s.I), "bwd_wu_q": (s.E * s.H, s.I)}
        buf = self.saved if name.startswith("bwd_") else self.fwd_scratch
        off = lay[name]
        if name == "pad_offsets":
            return buf[off:off + 4 * (s.E + 1)].view(torch.int32)
        if name.endswith("_sf"):
            base = name[:-3] + "_q"
            R, K = rows_k[base]
            seg, group = sf_grouping(base[4:] if base.startswith("bwd_") else base, s, Mp)
            return buf[off:off + sf_layout_bytes(R, K, seg, group)]
        R, K = rows_k[name]
        return buf[off:off + R * K].view(R, K)

    @_on_own_device
    def route(self, logits, stream=None):
        route(self.cfg, logits, self.routing, self.route_scratch, stream)

    @_on_own_device
    def forward(self, x, W_gate, W_up, W_down, out=None, stream=None, save=True):
        """save=False: a checkpointed layer's first pass (out only; call recompute
        before backward)."""
        if out is None:
            with _on_stream(stream):
                out = torch.empty((self.shape.T, self.shape.H), dtype=torch.int16, device=self.device)
        forward(self.cfg, x, self.routing, W_gate, W_up, W_down, out, self.saved, self.fwd_scratch, stream,
                save=save)
        return out

    @_on_own_device
    def recompute(self, x, W_gate, W_up, W_down, stream=None):
        """What backward reads, rebuilt from the same inputs (no out)."""
        forward_recompute(self.cfg, x, self.routing, W_gate, W_up, W_down, self.saved, self.fwd_scratch, stream)

    @_on_own_device
    def backward(self, dy, x, W_gate, W_up, W_down, grads=None, stream=None):
        s = self.shape
        dev = self.device
        if grads is None:
            with _on_stream(stream):
                grads = {
                    "dx": torch.empty((s.T, s.H), dtype=torch.int16, device=dev),
                    "dW_gate": torch.empty((s.E, s.H, s.I), dtype=torch.int16, device=dev),
                    "dW_up": torch.empty((s.E, s.H, s.I), dtype=torch.int16, device=dev),
                    "dW_down": torch.empty((s.E, s.I, s.H), dtype=torch.int16, device=dev),
                    "d_logits": torch.empty((s.T, s.E), dtype=torch.float32, device=dev),
                    "d_topk_w": torch.empty((s.T, s.k), dtype=torch.float32, device=dev),
                }
        backward(self.cfg, dy, x, self.routing, W_gate, W_up, W_down, self.saved, grads["dx"],
                 grads["dW_gate"], grads["dW_up"], grads["dW_down"], grads["d_logits"],
                 grads.get("d_topk_w"), self.bwd_scratch, stream)
        return grads

    @_on_own_device
    def status(self, stream=None) -> dict:
        return {n: get_device_status(b, stream) for n, b in
                (("route", self.route_scratch), ("forward", self.fwd_scratch), ("backward", self.bwd_scratch))}
