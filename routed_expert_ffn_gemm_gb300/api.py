"""Thin ctypes binding of libmoe_gb300.so (include/moe.h), same names.

Argument marshalling only: tensors become device pointers, the stream
defaults to torch's current stream, a non-zero status raises ``MoEError``.
Every step of the layer runs in the library's CUDA kernels; there is no
other implementation behind these functions.  The library is loaded on the
first call and a missing library is an error (build it with
``python -m routed_expert_ffn_gemm_gb300.build``).
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

# "fp8a8": FP8 weights with FP8 (per-row E4M3) gate/up activations;
# "mxfp4": OCP MX 4-bit block-scaled weights
DTYPE = {"f32": 0, "bf16": 1, "fp8": 2, "fp8a8": 3, "mxfp4": 4}
OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_DEVICE_TIMEOUT = -5
ERR_DEVICE_BOUNDS = -6


class moe_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "ffn", "E", "k", "ffn_shared", "act_dtype", "w_dtype")]


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} failed: {moe_status_string(status)}"
        if status == ERR_CUDA:
            msg += f" ({_lib().moe_last_cuda_error().decode()})"
        super().__init__(msg)


_LIB = None
_VP = ctypes.c_void_p
_PP = ctypes.POINTER(moe_problem)
_I, _L, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_float

_SIGS = {
    "moe_router_topk": [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_permute": [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP],
    "moe_grouped_swiglu": [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP],
    "moe_combine": [_PP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_layer_forward": [_PP] + [_VP] * 17 + [ctypes.c_size_t, _VP],
    "moe_workspace_size": [_PP, ctypes.POINTER(ctypes.c_size_t)],
    "moe_read_device_status": [_VP, ctypes.POINTER(ctypes.c_int32)],
    "moe_status_string": [ctypes.c_int32],
    "moe_last_cuda_error": [],
    "moe_abi_version": [],
    "moe_selftest_bounded_wait": [ctypes.c_int64, _VP],
    "moe_stage_timer_create": [ctypes.POINTER(_VP)],
    "moe_stage_timer_destroy": [_VP],
    "moe_stage_timer_read": [_VP, ctypes.POINTER(ctypes.c_float)],
    "moe_layer_forward_timed": [_PP] + [_VP] * 17 + [ctypes.c_size_t, _VP, _VP],
    "moe_layer_launch_count": [_PP, ctypes.POINTER(ctypes.c_int32)],
    "moe_plan_info": [_PP, ctypes.POINTER(ctypes.c_int32)],
    "moe_plan_info_for": [_PP, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
    "moe_layer_launch_count_for": [_PP, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
    "moe_workspace_size_for": [_PP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_permute_static_scratch": [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP],
    "moe_quantize_rows_e4m3": [ctypes.c_int32, ctypes.c_int32, _VP, _VP, _VP, _VP],
    "moe_split_rows_e4m3x2": [ctypes.c_int32, ctypes.c_int32, _VP, _VP, _VP, _VP],
    "moe_quantize_blocks_e4m3": [_I] * 4 + [_VP, _L, _VP, _VP, _VP],
    "moe_grouped_block_gemm": [_I] * 6 + [_VP] * 7,
    "moe_swiglu_save_e4m3": [_I, _I, _VP, _VP, _L] + [_VP] * 6,
    "moe_swiglu_backward_e4m3": [_I, _I] + [_VP] * 5 + [_L] + [_VP] * 4,
    "moe_grouped_wgrad": [_I] * 7 + [_VP, _L] + [_VP] * 5,
    "moe_router_losses": [_I] * 3 + [_VP] * 3 + [_F, _F] + [_VP] * 4 + [ctypes.c_size_t, _VP],
    "moe_router_losses_workspace_size": [_I, _I, ctypes.POINTER(ctypes.c_size_t)],
    "moe_router_losses_workspace_size_for": [_I, _I, _I, ctypes.POINTER(ctypes.c_size_t)],
    "moe_router_losses_backward": [_I] * 3 + [_VP] * 3 + [_F, _F] + [_VP] * 7,
    "moe_dispatch": [_I] * 7 + [_VP, _L] + [_VP] * 8 + [ctypes.c_size_t, _VP],
    "moe_dispatch_workspace_size": [_I, _I, _I, ctypes.POINTER(ctypes.c_size_t)],
    "moe_combine_rows": [_I] * 5 + [_VP] * 6,
    "moe_combine_rows_backward": [_I] * 5 + [_VP] * 7,
    "moe_quantize_mxfp4": [_I] * 5 + [_VP, _L] + [_VP] * 3,
    "moe_mxfp4_values": [_I] * 4 + [_VP] * 4,
    "moe_swiglu_mxfp4": [_I] * 3 + [_VP, _VP, _L] + [_VP] * 4,
    "moe_grouped_mxfp4_gemm": [_I] * 5 + [_VP] * 6 + [_L, _VP],
}
STAGES = ("router", "permute", "gate_up", "down", "shared", "combine")
EXPORTS = tuple(_SIGS)


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m routed_expert_ffn_gemm_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int32
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_last_cuda_error.restype = ctypes.c_char_p
        _LIB = lib
    return _LIB


def problem(T, d, ffn, E, k, ffn_shared=0, act="bf16", wfmt="bf16") -> moe_problem:
    return moe_problem(T, d, ffn, E, k, ffn_shared, DTYPE[act], DTYPE[wfmt])


def problem_of(shape) -> moe_problem:
    """moe_problem of an ``inputs.MoEShape``."""
    return problem(shape.T, shape.d, shape.ffn, shape.E, shape.k, shape.ffn_shared, shape.act, shape.wfmt)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the library takes device tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# Sizes checked before each call.  The C entry points take bare pointers,
# so a tensor smaller than the problem says, or of another element size,
# would be read or written out of bounds on the device; here it is a
# ValueError instead.  Null pointers, alignment and workspace sizes are the
# library's own checks.

def _check(t: Optional[torch.Tensor], name: str, elems: int, esize: int, dtype=None):
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, the call takes {dtype}")
    if t.element_size() != esize:
        raise ValueError(f"{name}: {t.element_size()}-byte elements, the problem needs {esize}-byte ones")
    if t.numel() < elems:
        raise ValueError(f"{name}: {t.numel()} elements, the problem needs {elems}")


def _act_size(p) -> int:
    return 4 if p.act_dtype == DTYPE["f32"] else 2


def _key(p) -> tuple:
    return (p.T, p.d, p.ffn, p.E, p.k, p.ffn_shared, p.act_dtype, p.w_dtype)


@functools.lru_cache(maxsize=256)
def _expert_reqs(key) -> tuple:
    """(name, elements, element size, dtype) of the routed expert weights
    and scales, per weight mode: gate/up [E, ffn, d], down [E, d, ffn]; FP8
    codes with fp32 scales [E, ffn] / [E, d]; MXFP4 codes two per byte with
    UE8M0 block scales [E, d/32, ffn] / [E, ffn/32, d]."""
    _, d, f, E, _, _, _, wdt = key
    if wdt == DTYPE["mxfp4"]:
        w, ws, gs, ds, ss = E * f * d // 2, 1, E * (d // 32) * f, E * (f // 32) * d, 1
    elif wdt in (DTYPE["fp8"], DTYPE["fp8a8"]):
        w, ws, gs, ds, ss = E * f * d, 1, E * f, E * d, 4
    else:
        w, ws, gs, ds, ss = E * f * d, 4 if wdt == DTYPE["f32"] else 2, 0, 0, 4
    return (("w_gate", w, ws, None), ("w_up", w, ws, None), ("w_down", w, ws, None),
            ("s_gate", gs, ss, None), ("s_up", gs, ss, None), ("s_down", ds, ss, None))


@functools.lru_cache(maxsize=256)
def _layer_reqs(key) -> tuple:
    T, d, _, E, k, fs, adt, _ = key
    a = 4 if adt == DTYPE["f32"] else 2
    return ((("x", T * d, a, None), ("w_router", E * d, a, None), ("router_bias", E, 4, torch.float32))
            + _expert_reqs(key)
            + (("w_shared_gate", fs * d, a, None), ("w_shared_up", fs * d, a, None),
               ("w_shared_down", fs * d, a, None), ("out", T * d, a, None),
               ("topk_idx_out", T * k, 4, torch.int32), ("topk_w_out", T * k, 4, torch.float32),
               ("counts_out", E, 4, torch.int32)))


def _verify(reqs, tensors):
    for t, (name, elems, esize, dtype) in zip(tensors, reqs):
        if t is not None and (t.numel() < elems or t.element_size() != esize
                              or (dtype is not None and t.dtype != dtype)):
            _check(t, name, elems, esize, dtype)


def _check_experts(p, w_gate, w_up, w_down, s_gate, s_up, s_down):
    _verify(_expert_reqs(_key(p)), (w_gate, w_up, w_down, s_gate, s_up, s_down))


def _check_layer(p, *tensors):
    """The 16 tensors of moe_layer_forward, x .. counts_out, in order."""
    _verify(_layer_reqs(_key(p)), tensors)


def _stream(stream):
    # (torch.cuda.current_stream() builds a Stream object: 10 us of host time
    # a call where a decode step's kernels take 5)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _on_stream(stream, fn, *args):
    """fn(*args) with `stream` current, for calls that allocate or copy: what
    they make is ordered with their kernels and not reused before those end.
    Results are also kept from reuse until the stream that is current here has
    done what it was given by the time they are dropped."""
    here = torch.cuda.current_stream()
    if stream.cuda_stream == here.cuda_stream:
        return fn(*args)
    given = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(given):
        out = fn(*args)
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, torch.Tensor):
            t.record_stream(here)
    return out


def _call(name, *args):
    st = getattr(_lib(), name)(*args)
    if st != OK:
        raise MoEError(name, st)


@functools.lru_cache(maxsize=None)
def _fn(name):
    return getattr(_lib(), name)


def _run(name, *args):
    """_call with the entry point looked up once (a quarter of a microsecond)."""
    st = _fn(name)(*args)
    if st != OK:
        raise MoEError(name, st)


def moe_router_topk(p, x, w_router, router_bias, logits_in, logits_out, topk_idx, topk_w, stream=None):
    a = _act_size(p)
    _check(x, "x", p.T * p.d, a)
    _check(w_router, "w_router", p.E * p.d, a)
    _check(router_bias, "router_bias", p.E, 4, torch.float32)
    _check(logits_in, "logits_in", p.T * p.E, 4, torch.float32)
    _check(logits_out, "logits_out", p.T * p.E, 4, torch.float32)
    _check(topk_idx, "topk_idx", p.T * p.k, 4, torch.int32)
    _check(topk_w, "topk_w", p.T * p.k, 4, torch.float32)
    _call("moe_router_topk", ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(router_bias),
          _ptr(logits_in), _ptr(logits_out), _ptr(topk_idx), _ptr(topk_w), _stream(stream))


def _check_permute(p, topk_idx, x, counts, offsets, perm_token, inv_row, x_perm):
    R, a = p.T * p.k, _act_size(p)
    _check(topk_idx, "topk_idx", R, 4, torch.int32)
    _check(x, "x", p.T * p.d, a)
    _check(counts, "counts", p.E, 4, torch.int32)
    _check(offsets, "offsets", p.E + 1, 4, torch.int32)
    _check(perm_token, "perm_token", R, 4, torch.int32)
    _check(inv_row, "inv_row", R, 4, torch.int32)
    _check(x_perm, "x_perm", R * p.d, a)


def moe_permute(p, topk_idx, x, counts, offsets, perm_token, inv_row, x_perm, workspace, stream=None):
    _check_permute(p, topk_idx, x, counts, offsets, perm_token, inv_row, x_perm)
    _call("moe_permute", ctypes.byref(p), _ptr(topk_idx), _ptr(x), _ptr(counts), _ptr(offsets),
          _ptr(perm_token), _ptr(inv_row), _ptr(x_perm), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))


def moe_permute_static_scratch(p, topk_idx, x, counts, offsets, perm_token, inv_row, x_perm, stream=None):
    """moe_permute for callers that cannot allocate device memory: the
    permutation's scratch comes from a fixed 1 MiB array inside the library
    instead of a caller workspace (see include/moe.h for its limits)."""
    _check_permute(p, topk_idx, x, counts, offsets, perm_token, inv_row, x_perm)
    _call("moe_permute_static_scratch", ctypes.byref(p), _ptr(topk_idx), _ptr(x), _ptr(counts),
          _ptr(offsets), _ptr(perm_token), _ptr(inv_row), _ptr(x_perm), _stream(stream))


def moe_grouped_swiglu(p, x_perm, offsets, w_gate, w_up, w_down, s_gate, s_up, s_down, y_perm,
                       workspace, stream=None):
    R, a = p.T * p.k, _act_size(p)
    _check(x_perm, "x_perm", R * p.d, a)
    _check(offsets, "offsets", p.E + 1, 4, torch.int32)
    _check_experts(p, w_gate, w_up, w_down, s_gate, s_up, s_down)
    _check(y_perm, "y_perm", R * p.d, a)
    _call("moe_grouped_swiglu", ctypes.byref(p), _ptr(x_perm), _ptr(offsets), _ptr(w_gate), _ptr(w_up),
          _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(y_perm), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))


def moe_quantize_rows_e4m3(x, codes, scales, stream=None):
    """Per-row E4M3 codes (uint8 [rows, cols]) and fp32 scales ([rows]) of
    bf16 rows x [rows, cols]."""
    rows, cols = (int(v) for v in x.shape)
    _check(x, "x", rows * cols, 2)
    _check(codes, "codes", rows * cols, 1)
    _check(scales, "scales", rows, 4, torch.float32)
    _call("moe_quantize_rows_e4m3", rows, cols, _ptr(x), _ptr(codes), _ptr(scales), _stream(stream))


def moe_split_rows_e4m3x2(x, codes, scales, stream=None):
    """bf16 rows x [rows, cols] as two E4M3 rows each: codes uint8
    [2, rows, cols] (every row's hi codes, then every row's lo codes) and
    power-of-two fp32 scales [rows], with x = s * (hi + lo)."""
    rows, cols = (int(v) for v in x.shape)
    _check(x, "x", rows * cols, 2)
    _check(codes, "codes", 2 * rows * cols, 1)
    _check(scales, "scales", rows, 4, torch.float32)
    _call("moe_split_rows_e4m3x2", rows, cols, _ptr(x), _ptr(codes), _ptr(scales), _stream(stream))


def moe_combine(p, y_perm, inv_row, topk_w, shared_out, out, stream=None):
    R, a = p.T * p.k, _act_size(p)
    _check(y_perm, "y_perm", R * p.d, a)
    _check(inv_row, "inv_row", R, 4, torch.int32)
    _check(topk_w, "topk_w", R, 4, torch.float32)
    _check(shared_out, "shared_out", p.T * p.d, a)
    _check(out, "out", p.T * p.d, a)
    _call("moe_combine", ctypes.byref(p), _ptr(y_perm), _ptr(inv_row), _ptr(topk_w), _ptr(shared_out),
          _ptr(out), _stream(stream))


def moe_layer_forward(p, x, w_router, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down,
                      w_shared_gate, w_shared_up, w_shared_down, out, topk_idx_out, topk_w_out,
                      counts_out, workspace, stream=None):
    _check_layer(p, x, w_router, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down, w_shared_gate,
                 w_shared_up, w_shared_down, out, topk_idx_out, topk_w_out, counts_out)
    _call("moe_layer_forward", ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(router_bias), _ptr(w_gate),
          _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(w_shared_gate),
          _ptr(w_shared_up), _ptr(w_shared_down), _ptr(out), _ptr(topk_idx_out), _ptr(topk_w_out),
          _ptr(counts_out), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))


def moe_layer_forward_timed(p, x, w_router, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down,
                            w_shared_gate, w_shared_up, w_shared_down, out, topk_idx_out, topk_w_out,
                            counts_out, workspace, timer, stream=None):
    _check_layer(p, x, w_router, router_bias, w_gate, w_up, w_down, s_gate, s_up, s_down, w_shared_gate,
                 w_shared_up, w_shared_down, out, topk_idx_out, topk_w_out, counts_out)
    _call("moe_layer_forward_timed", ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(router_bias),
          _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down),
          _ptr(w_shared_gate), _ptr(w_shared_up), _ptr(w_shared_down), _ptr(out), _ptr(topk_idx_out),
          _ptr(topk_w_out), _ptr(counts_out), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream),
          timer.handle)


class StageTimer:
    """moe_stage_timer: CUDA events between the stages of one layer call."""

    def __init__(self):
        h = ctypes.c_void_p(None)
        _call("moe_stage_timer_create", ctypes.byref(h))
        self.handle = h

    def read(self):
        """{stage: milliseconds} of the last timed call (waits for it)."""
        ms = (ctypes.c_float * len(STAGES))()
        _call("moe_stage_timer_read", self.handle, ms)
        return dict(zip(STAGES, (float(v) for v in ms)))

    def close(self):
        if self.handle is not None:
            _lib().moe_stage_timer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_layer_launch_count(p) -> int:
    n = ctypes.c_int32(0)
    _call("moe_layer_launch_count", ctypes.byref(p), ctypes.byref(n))
    return int(n.value)


def _plan_dict(info) -> dict:
    return {"bn_gateup": info[0], "bn_down": info[1], "splits_down": info[2], "grid": info[3],
            "splits_gateup": info[4], "pair_gateup": info[5] & 1, "pair_down": (info[5] >> 1) & 1}


def moe_plan_info(p) -> dict:
    info = (ctypes.c_int32 * 6)()
    _call("moe_plan_info", ctypes.byref(p), info)
    return _plan_dict(info)


def moe_workspace_size(p) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_workspace_size", ctypes.byref(p), ctypes.byref(n))
    return int(n.value)


# The planning answers for a device with `num_sms` SMs, computed on the host
# (no device needed).

def moe_plan_info_for(p, num_sms: int) -> dict:
    info = (ctypes.c_int32 * 6)()
    _call("moe_plan_info_for", ctypes.byref(p), int(num_sms), info)
    return _plan_dict(info)


def moe_layer_launch_count_for(p, num_sms: int) -> int:
    n = ctypes.c_int32(0)
    _call("moe_layer_launch_count_for", ctypes.byref(p), int(num_sms), ctypes.byref(n))
    return int(n.value)


def moe_workspace_size_for(p, num_sms: int) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_workspace_size_for", ctypes.byref(p), int(num_sms), ctypes.byref(n))
    return int(n.value)


def moe_read_device_status(stream=None) -> int:
    v = ctypes.c_int32(0)
    _call("moe_read_device_status", _stream(stream), ctypes.byref(v))
    return int(v.value)


def moe_status_string(status: int) -> str:
    return _lib().moe_status_string(int(status)).decode()


def moe_abi_version() -> int:
    return int(_lib().moe_abi_version())


def moe_selftest_bounded_wait(timeout_ns: int, stream=None):
    _call("moe_selftest_bounded_wait", int(timeout_ns), _stream(stream))


# ---------------------------------------------------------------------------
# conveniences over the C calls (allocation through torch)
# ---------------------------------------------------------------------------

def workspace_for(p, device="cuda") -> torch.Tensor:
    """A device workspace of moe_workspace_size(p) bytes (16-byte aligned)."""
    return torch.empty(max(16, moe_workspace_size(p)), dtype=torch.uint8, device=device)


def layer_forward(p, case, out=None, workspace=None, want_routing=False, stream=None, timer=None):
    """moe_layer_forward (or moe_layer_forward_timed when a StageTimer is
    given) on a case dict (``inputs.make_case`` keys)."""
    if stream is not None:
        return _on_stream(stream, layer_forward, p, case, out, workspace, want_routing, None, timer)
    x = case["x"]
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = workspace_for(p, x.device)
    idx = w = counts = None
    if want_routing:
        idx = torch.empty((p.T, p.k), dtype=torch.int32, device=x.device)
        w = torch.empty((p.T, p.k), dtype=torch.float32, device=x.device)
        counts = torch.empty((p.E,), dtype=torch.int32, device=x.device)
    args = (p, x, case["w_router"], case["router_bias"], case["w_gate"], case["w_up"],
            case["w_down"], case["s_gate"], case["s_up"], case["s_down"],
            case["w_shared_gate"], case["w_shared_up"], case["w_shared_down"], out,
            idx, w, counts, workspace)
    if timer is None:
        moe_layer_forward(*args)
    else:
        moe_layer_forward_timed(*args, timer)
    return (out, idx, w, counts) if want_routing else out


# ---------------------------------------------------------------------------
# training the routed experts in 8 bits
# ---------------------------------------------------------------------------

BLOCK = 128
SCALE = {"amax": 0, "pow2": 1}
_TYPES = {torch.float32: DTYPE["f32"], torch.bfloat16: DTYPE["bf16"]}


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _type(t, name: str) -> int:
    if t not in _TYPES:
        raise ValueError(f"{name}: {t}, the call takes float32 or bfloat16")
    return _TYPES[t]


def _exact(t: Optional[torch.Tensor], name: str, shape, dtype) -> None:
    if t is not None and (t.dtype is not dtype or t.shape != shape):
        raise ValueError(f"{name}: {t.dtype} {list(t.shape)}, the call takes {dtype} {list(shape)}")


def _rows(t: torch.Tensor, name: str, dtype=None) -> int:
    """The row pitch in elements of a matrix whose rows may lie apart."""
    shape = t.shape
    if len(shape) != 2 or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name}: {t.dtype} {list(shape)}, the call takes a matrix" + (f" of {dtype}" if dtype else ""))
    (rows, cols), (pitch, step) = shape, t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and pitch < cols):
        raise ValueError(f"{name}: the elements of a row must be adjacent and rows must not overlap")
    return pitch if rows > 1 else cols


def _pitched(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("the library takes device tensors")
    return t.data_ptr()


def quantize_blocks(x, scale="amax", codes=None, scales=None, stream=None):
    """moe_quantize_blocks_e4m3 of the rows of x [..., cols] (a matrix's rows
    may lie apart): (codes uint8 [..., cols], scales fp32 [..., blocks])."""
    if stream is not None:
        return _on_stream(stream, quantize_blocks, x, scale, codes, scales)
    if scale not in SCALE:
        raise ValueError(f"scale: {scale!r}, the call takes {sorted(SCALE)}")
    kind, shape, dev = _type(x.dtype, "x"), x.shape, x.device
    cols = shape[-1]
    m = x if len(shape) == 2 else x.reshape(-1, cols)
    ld, sshape = _rows(m, "x"), (*shape[:-1], _blocks(cols))
    if codes is None:
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    else:
        _exact(codes, "codes", shape, torch.uint8)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.float32, device=dev)
    else:
        _exact(scales, "scales", sshape, torch.float32)
    _call("moe_quantize_blocks_e4m3", m.shape[0], cols, kind, SCALE[scale], _pitched(m), ld, _ptr(codes), _ptr(scales),
          _stream(None))
    return codes, scales


def grouped_block_gemm(a, a_scales, offsets, w, w_scales, transposed=False, out_dtype=torch.bfloat16, out=None,
                       stream=None):
    """moe_grouped_block_gemm: rows a [R, K] (codes) of each expert times its
    w [E, N, K] (transposed: [E, K, N]) -> [R, N]."""
    if stream is not None:
        return _on_stream(stream, grouped_block_gemm, a, a_scales, offsets, w, w_scales, transposed, out_dtype, out)
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a: [R, K] and w: [E, N, K] are expected")
    R, K = a.shape
    E, N, Kw = (w.shape[0], w.shape[2], w.shape[1]) if transposed else w.shape
    if K != Kw:
        raise ValueError(f"w: {list(w.shape)} does not reduce over {K} columns")
    kind = _type(out_dtype if out is None else out.dtype, "out")
    out = torch.empty((R, N), dtype=out_dtype, device=a.device) if out is None else out
    sshape = (E, _blocks(K), _blocks(N)) if transposed else (E, _blocks(N), _blocks(K))
    _exact(a, "a", (R, K), torch.uint8)
    _exact(a_scales, "a_scales", (R, _blocks(K)), torch.float32)
    _exact(offsets, "offsets", (E + 1,), torch.int32)
    _exact(w, "w", w.shape, torch.uint8)
    _exact(w_scales, "w_scales", sshape, torch.float32)
    _exact(out, "out", (R, N), out.dtype)
    _call("moe_grouped_block_gemm", R, K, N, E, int(bool(transposed)), kind, _ptr(a), _ptr(a_scales), _ptr(offsets),
          _ptr(w), _ptr(w_scales), _ptr(out), _stream(None))
    return out


class SwigluSaved(NamedTuple):
    """What swiglu_save returns: h (bf16) and its codes and scales where asked
    for, and g and u as kept for the backward pass."""
    h: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    saved: torch.Tensor
    saved_scales: torch.Tensor


class SwigluGrads(NamedTuple):
    """What swiglu_backward returns: dg | du [R, 2 ffn], h again and the codes
    and scales of dg | du where asked for."""
    d_gu: torch.Tensor
    h: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def swiglu_save(g, u, want_h=False, want_codes=True, stream=None) -> SwigluSaved:
    """moe_swiglu_save_e4m3 of g and u [R, ffn] bf16 (for instance the halves
    of one product's rows)."""
    if stream is not None:
        return _on_stream(stream, swiglu_save, g, u, want_h, want_codes)
    ld = _rows(g, "g", torch.bfloat16)
    if _rows(u, "u", torch.bfloat16) != ld or u.shape != g.shape:
        raise ValueError("g and u: two matrices of one shape and row pitch are expected")
    (R, f), dev, nb = g.shape, g.device, _blocks(g.shape[1])
    h = torch.empty((R, f), dtype=torch.bfloat16, device=dev) if want_h else None
    codes = torch.empty((R, f), dtype=torch.uint8, device=dev) if want_codes else None
    scales = torch.empty((R, nb), dtype=torch.float32, device=dev) if want_codes else None
    saved = torch.empty((2, R, f), dtype=torch.uint8, device=dev)
    saved_scales = torch.empty((2, R, nb), dtype=torch.float32, device=dev)
    _call("moe_swiglu_save_e4m3", R, f, _pitched(g), _pitched(u), ld, _ptr(h), _ptr(codes), _ptr(scales), _ptr(saved),
          _ptr(saved_scales), _stream(None))
    return SwigluSaved(h, codes, scales, saved, saved_scales)


def swiglu_backward(saved, saved_scales, dh, want_h=False, want_codes=False, stream=None) -> SwigluGrads:
    """moe_swiglu_backward_e4m3 of what swiglu_save kept and dh [R, ffn] bf16."""
    if stream is not None:
        return _on_stream(stream, swiglu_backward, saved, saved_scales, dh, want_h, want_codes)
    if dh.dim() != 2:
        raise ValueError("dh: [R, ffn] is expected")
    R, f = dh.shape
    _exact(dh, "dh", (R, f), torch.bfloat16)
    _exact(saved, "saved", (2, R, f), torch.uint8)
    _exact(saved_scales, "saved_scales", (2, R, _blocks(f)), torch.float32)
    d_gu = torch.empty((R, 2 * f), dtype=torch.bfloat16, device=dh.device)
    h = torch.empty((R, f), dtype=torch.bfloat16, device=dh.device) if want_h else None
    codes = torch.empty((R, 2 * f), dtype=torch.uint8, device=dh.device) if want_codes else None
    scales = torch.empty((R, _blocks(2 * f)), dtype=torch.float32, device=dh.device) if want_codes else None
    dg = _ptr(d_gu)
    _call("moe_swiglu_backward_e4m3", R, f, _ptr(saved), _ptr(saved_scales), _ptr(dh), dg,
          dg + 2 * f if dg else None, 2 * f, _ptr(h), _ptr(codes), _ptr(scales), _stream(None))
    return SwigluGrads(d_gu, h, codes, scales)


def grouped_wgrad(dy, x, x_scales, offsets, dw=None, accumulate=False, dw_dtype=torch.float32, stream=None):
    """moe_grouped_wgrad: dw [E, N, K] of dy [R, N] bf16 (its rows may lie
    apart) and x [R, K], bf16 (x_scales None) or codes with their scales."""
    if stream is not None:
        return _on_stream(stream, grouped_wgrad, dy, x, x_scales, offsets, dw, accumulate, dw_dtype)
    ld = _rows(dy, "dy", torch.bfloat16)
    R, N = dy.shape
    K, E = x.shape[-1], offsets.numel() - 1
    _exact(x, "x", (R, K), torch.bfloat16 if x_scales is None else torch.uint8)
    _exact(x_scales, "x_scales", (R, _blocks(K)), torch.float32)
    _exact(offsets, "offsets", (E + 1,), torch.int32)
    if dw is None:
        if accumulate:
            raise ValueError("dw: accumulating needs the tensor to add to")
        dw = torch.empty((E, N, K), dtype=dw_dtype, device=dy.device)
    kind = _type(dw.dtype, "dw")
    _exact(dw, "dw", (E, N, K), dw.dtype)
    _call("moe_grouped_wgrad", R, N, K, E, DTYPE["bf16" if x_scales is None else "fp8"], kind, int(bool(accumulate)),
          _pitched(dy), ld, _ptr(x), _ptr(x_scales), _ptr(offsets), _ptr(dw), _stream(None))
    return dw


class RouterLosses(NamedTuple):
    """What router_losses returns: loss [2] (balance, z), counts [E + 1] (the
    experts', then the unmasked tokens), lse [T], and the coefficients."""
    loss: torch.Tensor
    counts: torch.Tensor
    lse: torch.Tensor
    balance: float
    z: float


@functools.lru_cache(maxsize=256)
def _router_workspace(T: int, E: int, device: int) -> int:
    return moe_router_losses_workspace_size(T, E)


def moe_router_losses_workspace_size(T: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_router_losses_workspace_size", T, E, ctypes.byref(n))
    return int(n.value)


def moe_router_losses_workspace_size_for(T: int, E: int, num_sms: int) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_router_losses_workspace_size_for", T, E, num_sms, ctypes.byref(n))
    return int(n.value)


def _check_router(logits, idx, mask):
    if logits.dim() != 2 or idx.dim() != 2:
        raise ValueError("logits: [T, E] and topk_idx: [T, k] are expected")
    T, E = logits.shape
    k = idx.shape[1]
    _exact(logits, "logits", (T, E), torch.float32)
    _exact(idx, "topk_idx", (T, k), torch.int32)
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (T,)):
        raise ValueError(f"mask: {mask.dtype} {list(mask.shape)}, the call takes bool or uint8 [{T}]")
    return T, E, k


def router_losses(logits, topk_idx, balance, z, mask=None, workspace=None, stream=None) -> RouterLosses:
    """moe_router_losses of logits [T, E] and the chosen experts [T, k]."""
    if stream is not None:
        return _on_stream(stream, router_losses, logits, topk_idx, balance, z, mask, workspace)
    T, E, k = _check_router(logits, topk_idx, mask)
    dev = logits.device
    loss = torch.empty(2, dtype=torch.float32, device=dev)
    counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(_router_workspace(T, E, torch._C._cuda_getDevice()), dtype=torch.uint8, device=dev)
    _call("moe_router_losses", T, E, k, _ptr(logits), _ptr(topk_idx), _ptr(mask), balance, z, _ptr(loss), _ptr(counts),
          _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(None))
    return RouterLosses(loss, counts, lse, balance, z)


def router_losses_backward(logits, topk_idx, losses: RouterLosses, grad=None, topk_w=None, d_topk_w=None, mask=None,
                           stream=None):
    """moe_router_losses_backward: the gradient of the logits [T, E]; grad is
    a device scalar (None: 1)."""
    if stream is not None:
        return _on_stream(stream, router_losses_backward, logits, topk_idx, losses, grad, topk_w, d_topk_w, mask)
    T, E, k = _check_router(logits, topk_idx, mask)
    _exact(losses.counts, "counts", (E + 1,), torch.int32)
    _exact(losses.lse, "lse", (T,), torch.float32)
    _check(grad, "grad", 1, 4, torch.float32)
    _exact(topk_w, "topk_w", (T, k), torch.float32)
    _exact(d_topk_w, "d_topk_w", (T, k), torch.float32)
    d_logits = torch.empty_like(logits)
    _call("moe_router_losses_backward", T, E, k, _ptr(logits), _ptr(topk_idx), _ptr(mask), losses.balance, losses.z,
          _ptr(losses.counts), _ptr(losses.lse), _ptr(grad), _ptr(topk_w), _ptr(d_topk_w), _ptr(d_logits),
          _stream(None))
    return d_logits


# ---------------------------------------------------------------------------
# the experts in 4 bits, and the gradients of the token movement
# ---------------------------------------------------------------------------

MX_BLOCK = 32
MX_SCALE = {"floor": 0, "fit": 1}


def _mx_scale(kind) -> int:
    if kind not in MX_SCALE:
        raise ValueError(f"scale: {kind!r}, the call takes {sorted(MX_SCALE)}")
    return MX_SCALE[kind]


def _here(t: torch.Tensor, *more) -> None:
    """The tensors are on the current device: the kernels run there."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the library takes device tensors")
    for o in more:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and {o.device}")
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"tensors on {t.device}, which is not the current device")


def _at(t: Optional[torch.Tensor]):
    """The address of a tensor that _here has seen."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


class Dispatched(NamedTuple):
    """What dispatch returns: the rows [T * k, d] (codes [T * k, d / 2] with
    scales [T * k, d / 32] where quantised), offsets [E + 1], counts [E],
    row_token [T * k] and inv_row [T, k]."""
    rows: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    offsets: torch.Tensor
    counts: torch.Tensor
    row_token: torch.Tensor
    inv_row: torch.Tensor


class CombineGrads(NamedTuple):
    """What combine_backward returns: the gradients of the rows and of the
    routing weights, None where not asked for."""
    dy: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]


class MxSwiglu(NamedTuple):
    """What swiglu_mxfp4 returns: h as codes [R, ffn / 2] and scales [R, ffn /
    32], and in bf16 where asked for."""
    codes: torch.Tensor
    scales: torch.Tensor
    h: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)
def moe_dispatch_workspace_size(T: int, E: int, k: int) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_dispatch_workspace_size", T, E, k, ctypes.byref(n))
    return int(n.value)


def _slots(idx, name) -> tuple:
    shape = idx.shape
    if len(shape) != 2 or idx.dtype is not torch.int32:
        raise ValueError(f"{name}: {idx.dtype} {list(shape)}, the call takes torch.int32 [T, k]")
    return shape


def dispatch(x, topk_idx, E, quantize=None, rows=None, scales=None, workspace=None, stream=None) -> Dispatched:
    """moe_dispatch of x [T, d] (its rows may lie apart) by topk_idx [T, k],
    negative where an assignment is dropped: rows of x's type, or MXFP4 with
    quantize "floor" or "fit".  x None: the maps alone."""
    if stream is not None:
        return _on_stream(stream, dispatch, x, topk_idx, E, quantize, rows, scales, workspace)
    T, k = _slots(topk_idx, "topk_idx")
    R, dev, empty = T * k, topk_idx.device, torch.empty
    size = moe_dispatch_workspace_size(T, E, k)  # (refuses sizes)
    if x is None:
        if quantize is not None or rows is not None or scales is not None:
            raise ValueError("rows: there are none without x")
        d, ld, kind, out_kind, mx, at = 8, 8, 1, 1, 0, None
    else:
        ld, kind, at, mx = _rows(x, "x"), _type(x.dtype, "x"), x.data_ptr(), 0
        n, d = x.shape
        if n != T:
            raise ValueError(f"x: {[n, d]}, topk_idx has {T} tokens")
        shape, t, out_kind = (R, d), x.dtype, kind
        if quantize is not None:
            if d % MX_BLOCK:
                raise ValueError(f"x: {d} columns are no multiple of {MX_BLOCK}")
            shape, t, out_kind, mx = (R, d // 2), torch.uint8, DTYPE["mxfp4"], _mx_scale(quantize)
            _exact(scales, "scales", (R, d // MX_BLOCK), torch.uint8)
        elif scales is not None:
            raise ValueError("scales: there are none without quantize")
        _exact(rows, "rows", shape, t)
    _here(topk_idx, x, rows, scales, workspace)
    if x is not None:
        if rows is None:
            rows = empty(shape, dtype=t, device=dev)
        if scales is None and quantize is not None:
            scales = empty((R, d // MX_BLOCK), dtype=torch.uint8, device=dev)
    # (four allocations: one with four views of it takes 6 us of host time more)
    offsets = empty(E + 1, dtype=torch.int32, device=dev)
    counts = empty(E, dtype=torch.int32, device=dev)
    row_token = empty(R, dtype=torch.int32, device=dev)
    inv_row = torch.empty_like(topk_idx, memory_format=torch.contiguous_format)
    if workspace is None:
        if size:
            workspace = empty(size, dtype=torch.uint8, device=dev)
    else:
        size = workspace.numel() * workspace.element_size()
    _run("moe_dispatch", T, d, E, k, kind, out_kind, mx, at, ld, _at(topk_idx), counts.data_ptr(), offsets.data_ptr(),
         row_token.data_ptr(), inv_row.data_ptr(), _at(rows), _at(scales), _at(workspace), size, _stream(None))
    return Dispatched(rows, scales, offsets, counts, row_token, inv_row)


def combine(y, inv_row, topk_w=None, add=None, out=None, stream=None):
    """moe_combine_rows: rows y [R, d] weighted (topk_w None: ones), summed
    back to tokens and added to add [T, d] -> [T, d]."""
    if stream is not None:
        return _on_stream(stream, combine, y, inv_row, topk_w, add, out)
    T, k = _slots(inv_row, "inv_row")
    if y.dim() != 2:
        raise ValueError("y: [R, d] is expected")
    _here(y, inv_row, topk_w, add, out)
    (R, d), dtype = y.shape, y.dtype
    kind = _type(dtype, "y")
    _exact(topk_w, "topk_w", (T, k), torch.float32)
    _exact(add, "add", (T, d), dtype)
    if out is None:
        out = torch.empty((T, d), dtype=dtype, device=y.device)
    else:
        _exact(out, "out", (T, d), dtype)
    _run("moe_combine_rows", T, d, k, R, kind, _at(y), _at(inv_row), _at(topk_w), _at(add), _at(out), _stream(None))
    return out


def dispatch_backward(d_rows, inv_row, add=None, out=None, stream=None):
    """The gradient of dispatch's x from its rows' d_rows [R, d], added to add
    [T, d] (what reaches x another way)."""
    return combine(d_rows, inv_row, None, add, out, stream)


def combine_backward(d_out, y, inv_row, topk_w=None, want_dy=True, want_dw=True, dy=None, stream=None) -> CombineGrads:
    """moe_combine_rows_backward: the gradients of combine's y and topk_w from
    d_out [T, d].  Rows that no assignment has stay as they are in dy."""
    if stream is not None:
        return _on_stream(stream, combine_backward, d_out, y, inv_row, topk_w, want_dy, want_dw, dy)
    T, k = _slots(inv_row, "inv_row")
    if y.dim() != 2:
        raise ValueError("y: [R, d] is expected")
    _here(y, d_out, inv_row, topk_w, dy)
    (R, d), dtype = y.shape, y.dtype
    kind = _type(dtype, "y")
    _exact(d_out, "d_out", (T, d), dtype)
    _exact(topk_w, "topk_w", (T, k), torch.float32)
    if dy is not None:
        _exact(dy, "dy", (R, d), dtype)
    elif want_dy:
        dy = torch.empty((R, d), dtype=dtype, device=y.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=y.device) if want_dw else None
    _run("moe_combine_rows_backward", T, d, k, R, kind, _at(d_out), _at(y), _at(inv_row), _at(topk_w), _at(dy), _at(dw),
         _stream(None))
    return CombineGrads(dy, dw)


@functools.lru_cache(maxsize=256)
def _mx_shapes(shape, weights: bool) -> tuple:
    """Rows, columns, rows of a weight matrix (0: none) and the shapes of codes
    and scales of values of this shape."""
    if weights and len(shape) != 3:
        raise ValueError(f"weights: {list(shape)}, the call takes [E, N, K]")
    cols = shape[-1]
    if cols % MX_BLOCK:
        raise ValueError(f"{cols} columns are no multiple of {MX_BLOCK}")
    rows, blocks = 1, cols // MX_BLOCK
    for n in shape[:-1]:
        rows *= n
    codes = torch.Size((*shape[:-1], cols // 2))
    if weights:
        return rows, cols, shape[1], codes, torch.Size((shape[0], blocks, shape[1]))
    return rows, cols, 0, codes, torch.Size((*shape[:-1], blocks))


def quantize_mxfp4(x, scale="floor", weights=False, codes=None, scales=None, stream=None):
    """moe_quantize_mxfp4 of x [..., cols] (a matrix's rows may lie apart):
    (codes uint8 [..., cols / 2], scales uint8 [..., cols / 32]); with weights
    of x [E, N, K], scales [E, K / 32, N] as the products take them.  Of a view
    that is no such matrix, a transposed one for instance, torch makes a copy
    first."""
    if stream is not None:
        return _on_stream(stream, quantize_mxfp4, x, scale, weights, codes, scales)
    mx, kind, shape, dev = _mx_scale(scale), _type(x.dtype, "x"), x.shape, x.device
    rows, cols, matrix, cshape, sshape = _mx_shapes(shape, weights)
    m = x if len(shape) == 2 else x.reshape(rows, cols)
    ld = _rows(m, "x")
    _here(x, codes, scales)
    if codes is None:
        codes = torch.empty(cshape, dtype=torch.uint8, device=dev)
    else:
        _exact(codes, "codes", cshape, torch.uint8)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.uint8, device=dev)
    else:
        _exact(scales, "scales", sshape, torch.uint8)
    _run("moe_quantize_mxfp4", rows, cols, kind, mx, matrix, m.data_ptr(), ld, _at(codes), _at(scales), _stream(None))
    return codes, scales


def mxfp4_values(codes, scales, dtype=torch.bfloat16, weights=False, out=None, stream=None):
    """moe_mxfp4_values: what quantize_mxfp4's codes and scales stand for."""
    if stream is not None:
        return _on_stream(stream, mxfp4_values, codes, scales, dtype, weights, out)
    shape = torch.Size((*codes.shape[:-1], 2 * codes.shape[-1]))
    rows, cols, matrix, cshape, sshape = _mx_shapes(shape, weights)
    _here(codes, scales, out)
    kind = _type(dtype if out is None else out.dtype, "out")
    _exact(codes, "codes", cshape, torch.uint8)
    _exact(scales, "scales", sshape, torch.uint8)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=codes.device)
    else:
        _exact(out, "out", shape, out.dtype)
    _run("moe_mxfp4_values", rows, cols, kind, matrix, _at(codes), _at(scales), _at(out), _stream(None))
    return out


def swiglu_mxfp4(g, u, scale="floor", want_h=False, stream=None) -> MxSwiglu:
    """moe_swiglu_mxfp4 of g and u [R, ffn] bf16 (for instance the halves of
    one product's rows)."""
    if stream is not None:
        return _on_stream(stream, swiglu_mxfp4, g, u, scale, want_h)
    mx, ld, shape = _mx_scale(scale), _rows(g, "g", torch.bfloat16), g.shape
    if _rows(u, "u", torch.bfloat16) != ld or u.shape != shape:
        raise ValueError("g and u: two matrices of one shape and row pitch are expected")
    _here(g, u)
    R, f, _, cshape, sshape = _mx_shapes(shape, False)
    dev = g.device
    codes = torch.empty(cshape, dtype=torch.uint8, device=dev)
    scales = torch.empty(sshape, dtype=torch.uint8, device=dev)
    h = torch.empty(shape, dtype=torch.bfloat16, device=dev) if want_h else None
    _run("moe_swiglu_mxfp4", R, f, mx, g.data_ptr(), u.data_ptr(), ld, codes.data_ptr(), scales.data_ptr(), _at(h),
         _stream(None))
    return MxSwiglu(codes, scales, h)


def grouped_mxfp4_gemm(a, a_scales, offsets, w, w_scales, out_dtype=torch.bfloat16, out=None, stream=None):
    """moe_grouped_mxfp4_gemm: MXFP4 rows a [R, K / 2] with scales [R, K / 32]
    of each expert times its w [E, N, K / 2] with scales [E, K / 32, N] -> [R,
    N] (out's rows may lie apart)."""
    if stream is not None:
        return _on_stream(stream, grouped_mxfp4_gemm, a, a_scales, offsets, w, w_scales, out_dtype, out)
    ashape, wshape, u8 = a.shape, w.shape, torch.uint8
    if len(ashape) != 2 or len(wshape) != 3 or ashape[1] != wshape[2]:
        raise ValueError(f"a: {list(ashape)} and w: {list(wshape)}, the call takes [R, K / 2] and [E, N, K / 2]")
    _here(a, a_scales, offsets, w, w_scales, out)
    (R, half), (E, N, _) = ashape, wshape
    K = 2 * half
    if K % MX_BLOCK:
        raise ValueError(f"a: {K} columns are no multiple of {MX_BLOCK}")
    _exact(a, "a", ashape, u8)
    _exact(a_scales, "a_scales", (R, K // MX_BLOCK), u8)
    _exact(offsets, "offsets", (E + 1,), torch.int32)
    _exact(w, "w", wshape, u8)
    _exact(w_scales, "w_scales", (E, K // MX_BLOCK, N), u8)
    if out is None:
        out = torch.empty((R, N), dtype=out_dtype, device=a.device)
    elif out.shape != (R, N):
        raise ValueError(f"out: {list(out.shape)}, the call takes {[R, N]}")
    kind = _type(out.dtype, "out")
    _run("moe_grouped_mxfp4_gemm", R, K, N, E, kind, _at(a), _at(a_scales), _at(offsets), _at(w), _at(w_scales),
         out.data_ptr(), _rows(out, "out"), _stream(None))
    return out
