"""Refusals and allocations of the 4-bit operators and the token movement,
without a GPU: the C entry points' argument checks answer before anything is
enqueued, the binding's checks raise before a pointer is taken, and what a call
with stream= makes belongs to that stream."""

import ctypes
import os
import re

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests.test_expert_training_checks import check
from tests.test_kernel_sources import text_of
from tests.test_stream_allocations import SIDE, Recorder

INV, UNS, WS, OK = api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED, api.ERR_WORKSPACE, api.OK
P = ctypes.c_void_p(0x1000)   # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned
BF16, F32, MX = 1, 0, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api._lib()


def test_dispatch(lib):
    good = dict(T=4, d=64, E=8, k=2, x_dtype=BF16, rows_dtype=BF16, kind=0, x=P, ld=64, idx=P, counts=P, offsets=P,
                token=P, inv=P, rows=P, scales=P, ws=None, size=0)
    check(lib.moe_dispatch, good, [
        (dict(T=-1), INV), (dict(d=0), INV), (dict(d=12, ld=16), UNS), (dict(E=0), INV), (dict(E=1025), UNS), (dict(k=0), INV),
        (dict(k=33), UNS), (dict(T=1 << 24), UNS), (dict(x_dtype=2), UNS), (dict(rows_dtype=F32), UNS), (dict(rows_dtype=2), UNS),
        (dict(rows_dtype=MX, d=40, ld=40), UNS), (dict(rows_dtype=MX, scales=None), INV), (dict(kind=2), INV), (dict(ld=56), INV),
        (dict(ld=68), INV), (dict(x=None), INV), (dict(idx=None), INV), (dict(counts=None), INV), (dict(offsets=None), INV),
        (dict(token=None), INV), (dict(inv=None), INV)]
        + [({n: ODD}, INV) for n in ("x", "idx", "counts", "offsets", "token", "inv", "rows", "scales")]
        + [(dict(T=4000), WS), (dict(T=4000, ws=P, size=16), WS), (dict(T=4000, ws=ODD, size=1 << 20), INV)])
    n = ctypes.c_size_t(7)
    assert lib.moe_dispatch_workspace_size(64, 256, 8, ctypes.byref(n)) == OK and n.value == 0
    assert lib.moe_dispatch_workspace_size(4000, 8, 2, ctypes.byref(n)) == OK and n.value > 0
    assert lib.moe_dispatch_workspace_size(4000, 8, 2, None) == INV
    assert lib.moe_dispatch_workspace_size(-1, 8, 2, ctypes.byref(n)) == INV
    assert lib.moe_dispatch_workspace_size(4, 0, 2, ctypes.byref(n)) == INV
    assert lib.moe_dispatch_workspace_size(4, 2000, 2, ctypes.byref(n)) == UNS


def test_combine(lib):
    good = dict(T=4, d=64, k=2, R=8, dtype=BF16, rows=P, inv=P, w=P, add=P, out=P)
    check(lib.moe_combine_rows, good, [
        (dict(T=-1), INV), (dict(d=0), INV), (dict(d=20), UNS), (dict(k=0), INV), (dict(k=40), UNS), (dict(R=-1), INV),
        (dict(R=(1 << 24) + 1), UNS), (dict(dtype=2), UNS), (dict(rows=None), INV), (dict(inv=None), INV), (dict(out=None), INV),
        (dict(T=0, rows=None, inv=None, out=None), OK)] + [({n: ODD}, INV) for n in ("rows", "inv", "w", "add", "out")])
    good = dict(T=4, d=64, k=2, R=8, dtype=F32, d_out=P, rows=P, inv=P, w=P, dr=P, dw=P)
    check(lib.moe_combine_rows_backward, good, [
        (dict(T=-1), INV), (dict(d=4), UNS), (dict(k=33), UNS), (dict(R=-2), INV), (dict(dtype=4), UNS), (dict(d_out=None), INV),
        (dict(inv=None), INV), (dict(rows=None), INV), (dict(dr=None, dw=None), OK), (dict(T=0, d_out=None), OK)]
        + [({n: ODD}, INV) for n in ("d_out", "rows", "inv", "w", "dr", "dw")])


def test_quantize_and_values(lib):
    good = dict(rows=32, cols=64, dtype=BF16, kind=0, matrix=0, x=P, ld=64, codes=P, scales=P)
    bad = [(dict(rows=-1), INV), (dict(cols=0), UNS), (dict(cols=48), UNS), (dict(dtype=2), UNS), (dict(matrix=-16), INV),
           (dict(matrix=24), INV), (dict(rows=(1 << 24) + 1), UNS), (dict(codes=None), INV),
           (dict(scales=None), INV), (dict(codes=ODD), INV), (dict(scales=ODD), INV)]
    check(lib.moe_quantize_mxfp4, good, bad + [
        (dict(kind=2), INV), (dict(ld=32), INV), (dict(ld=68), INV), (dict(x=None), INV), (dict(x=ODD), INV),
        (dict(rows=0, x=None, codes=None), OK)])
    good = dict(rows=32, cols=64, dtype=F32, matrix=0, codes=P, scales=P, out=P)
    check(lib.moe_mxfp4_values, good, bad + [(dict(out=None), INV), (dict(out=ODD), INV), (dict(rows=0, codes=None), OK)])


def test_swiglu(lib):
    good = dict(R=4, f=64, kind=1, g=P, u=P, ld=128, codes=P, scales=P, h=P)
    check(lib.moe_swiglu_mxfp4, good, [
        (dict(R=-1), INV), (dict(f=0), UNS), (dict(f=80), UNS), (dict(kind=-1), INV), (dict(ld=32), INV), (dict(ld=132), INV),
        (dict(g=None), INV), (dict(u=None), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(R=0, g=None), OK)]
        + [({n: ODD}, INV) for n in ("g", "u", "codes", "scales", "h")])


def test_product(lib):
    good = dict(R=4, K=128, N=256, E=2, out_dtype=BF16, a=P, sa=P, off=P, w=P, sw=P, out=P, ld=256)
    check(lib.moe_grouped_mxfp4_gemm, good, [
        (dict(R=-1), INV), (dict(K=0), INV), (dict(N=-16), INV), (dict(E=0), INV), (dict(K=80), UNS), (dict(N=24), UNS),
        (dict(E=1025), UNS), (dict(out_dtype=2), UNS), (dict(ld=240), INV), (dict(ld=260), INV), (dict(R=(1 << 24) + 1), UNS),
        (dict(R=0, a=None, out=None), OK)]
        + [({n: None}, INV) for n in ("a", "sa", "off", "w", "sw", "out")]
        + [({n: ODD}, INV) for n in ("a", "sa", "off", "w", "sw", "out")])


# ---------------------------------------------------------------- the binding

def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def b16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(*s)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


CALLS = [
    (api.dispatch, dict(x=b16(6, 64), topk_idx=i32(6, 2), E=8)),
    (api.dispatch, dict(x=f32(3000, 64), topk_idx=i32(3000, 2), E=8, quantize="fit")),
    (api.combine, dict(y=b16(12, 64), inv_row=i32(6, 2), topk_w=f32(6, 2), add=b16(6, 64))),
    (api.dispatch_backward, dict(d_rows=b16(12, 64), inv_row=i32(6, 2), add=b16(6, 64))),
    (api.combine_backward, dict(d_out=b16(6, 64), y=b16(12, 64), inv_row=i32(6, 2), topk_w=f32(6, 2))),
    (api.quantize_mxfp4, dict(x=b16(6, 64))),
    (api.quantize_mxfp4, dict(x=f32(3, 2, 64).transpose(0, 1))),
    (api.quantize_mxfp4, dict(x=b16(3, 32, 64), scale="fit", weights=True)),
    (api.mxfp4_values, dict(codes=u8(6, 32), scales=u8(6, 2))),
    (api.mxfp4_values, dict(codes=u8(3, 32, 32), scales=u8(3, 2, 32), dtype=torch.float32, weights=True)),
    (api.swiglu_mxfp4, dict(g=b16(6, 64), u=b16(6, 64), want_h=True)),
    (api.grouped_mxfp4_gemm, dict(a=u8(6, 32), a_scales=u8(6, 2), offsets=i32(3), w=u8(2, 48, 32), w_scales=u8(2, 2, 48))),
]
IDS = [f"{i}-{fn.__name__}" for i, (fn, _) in enumerate(CALLS)]


@pytest.mark.parametrize("fn,good", CALLS, ids=IDS)
def test_binding_refuses_other_sizes_types_and_places(fn, good, lib):
    with pytest.raises(ValueError, match="device tensors"):
        fn(**good)
    for name, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        if name not in ("x", "d_rows", "y") and len(good) > 1:  # (any number of rows is a batch of its own there)
            with pytest.raises(ValueError):
                fn(**dict(good, **{name: t[..., :-1] if t.dim() > 1 else t[:-1]}))
        with pytest.raises(ValueError):
            fn(**dict(good, **{name: t.double()}))


class Elsewhere:
    """Stands in for a tensor on another device."""
    def __init__(self, dev):
        self.dev, self.device = dev, f"cuda:{dev}"

    def get_device(self):
        return self.dev


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    api._here(Elsewhere(0), None, Elsewhere(0))
    for bad in ((Elsewhere(1), Elsewhere(1)), (Elsewhere(0), None, Elsewhere(1)), (Elsewhere(1),)):
        with pytest.raises(ValueError, match="cuda:1"):
            api._here(*bad)


def test_binding_refuses_other_arguments(lib):
    with pytest.raises(ValueError, match="scale"):
        api.quantize_mxfp4(b16(2, 64), "amax")
    with pytest.raises(ValueError, match="scale"):
        api.dispatch(b16(6, 64), i32(6, 2), 8, quantize=True)
    with pytest.raises(ValueError, match="multiple"):
        api.quantize_mxfp4(b16(2, 48))
    with pytest.raises(ValueError, match="weights"):
        api.quantize_mxfp4(b16(32, 64), weights=True)
    with pytest.raises(ValueError, match="without"):
        api.dispatch(None, i32(6, 2), 8, quantize="fit")
    with pytest.raises(ValueError, match="tokens"):
        api.dispatch(b16(5, 64), i32(6, 2), 8)
    with pytest.raises(ValueError, match="adjacent"):
        api.quantize_mxfp4(b16(64, 32).T)
    with pytest.raises(ValueError, match="pitch"):
        api.swiglu_mxfp4(b16(6, 256)[:, :128], b16(6, 128))
    with pytest.raises(api.MoEError):
        api.dispatch(b16(6, 64), i32(6, 2), 0)
    with pytest.raises(ValueError):
        api.grouped_mxfp4_gemm(u8(6, 32), u8(6, 2), i32(3), u8(2, 48, 48), u8(2, 3, 48))


@pytest.mark.parametrize("fn,good", CALLS, ids=IDS)
def test_what_a_call_makes_belongs_to_its_stream(monkeypatch, fn, good, lib):
    r = Recorder(monkeypatch)
    monkeypatch.setattr(api, "_here", lambda *t: None)
    monkeypatch.setattr(api, "_run", lambda name, *args: r.launched.append((name, args[-1])))
    out = fn(**good, stream=SIDE)
    assert r.made and r.launched and all(s is SIDE for _, s in r.made + r.launched)
    tensors = [t for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)]
    assert tensors and all(any(t is k for k in r.kept) for t in tensors)


# ----------------------------------------- rules that no launch can show

@pytest.mark.parametrize("name", ["mxfp4_gemm.cu", "mxfp4_gemm_many.cu"])
def test_copying_warp_waits_for_the_last_arrivals(name):
    # the MMAs' commits arrive on a slot's barrier by themselves: the CTA whose
    # barrier it is has to see the last one of each slot before it may leave
    text = text_of(name)
    role = text[text.index("- copies (lane 0)\n"):text.index("MOE_ERR_DEVICE_TIMEOUT", text.index("- copies (lane 0)\n"))]
    loop, wait = role.index("for (int u = u_first"), r"mbar_wait_bounded\(\s*empty_bar\("
    after = role[role.index("__shfl_sync", loop):]  # behind the loop over the units
    assert len(re.findall(wait, role)) == 2 and len(re.findall(wait, after)) == 1


def test_warp_that_loads_row_scales_does_not_fence():
    text = text_of("mxfp4_gemm.cuh")
    role = text[text.index("bool row_scales("):text.index("}  // namespace mx_gemm")]
    assert "__ldg" in text and "fence" not in re.sub(r"//.*", "", role)


def test_wait_limit_grows_with_the_work():
    limits = re.findall(r"wait_limit_ns\((.*?)\)", text_of("fp4_api.cu"))
    assert limits and all(all(v in a for v in "RNKE") for a in limits)


def test_kernel_sources_are_built():
    names = {os.path.basename(s) for s in build.sources()}
    assert {"dispatch.cu", "combine_rows.cu", "mxfp4.cu", "mxfp4_gemm.cu", "mxfp4_gemm_many.cu", "fp4_api.cu"} <= names
