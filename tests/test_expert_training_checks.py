"""Refusals of the expert-training operators, without a GPU: the C entry
points' argument checks answer before anything is enqueued, and the binding's
checks raise before a pointer is taken."""

import ctypes

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build

INV, UNS, WS, OK = api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED, api.ERR_WORKSPACE, api.OK
P = ctypes.c_void_p(0x1000)   # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api._lib()


def check(fn, good, cases):
    for change, want in cases:
        args = dict(good, **change)
        assert fn(*args.values(), None) == want, change


def test_quantize_blocks(lib):
    good = dict(rows=4, cols=128, dtype=1, kind=0, x=P, ld=128, codes=P, scales=P)
    check(lib.moe_quantize_blocks_e4m3, good, [
        (dict(rows=-1), INV), (dict(cols=0), UNS), (dict(cols=12), UNS), (dict(dtype=2), UNS), (dict(kind=2), INV),
        (dict(ld=120), INV), (dict(ld=132), INV), (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV),
        (dict(x=ODD), INV), (dict(codes=ODD), INV), (dict(rows=0, x=None, codes=None, scales=None), OK),
        (dict(rows=(1 << 24) + 1), UNS)])


def test_block_gemm(lib):
    good = dict(R=4, K=128, N=256, E=2, t=0, out_dtype=1, a=P, sa=P, off=P, w=P, sw=P, out=P)
    check(lib.moe_grouped_block_gemm, good, [
        (dict(R=-1), INV), (dict(K=0), INV), (dict(N=-16), INV), (dict(E=0), INV), (dict(K=120), UNS), (dict(N=24), UNS),
        (dict(E=1025), UNS), (dict(out_dtype=2), UNS), (dict(R=0, a=None, out=None), OK)]
        + [({n: None}, INV) for n in ("a", "sa", "off", "w", "sw", "out")]
        + [({n: ODD}, INV) for n in ("a", "sa", "off", "w", "sw", "out")])


def test_swiglu_save(lib):
    good = dict(R=4, f=128, g=P, u=P, ld=128, h=P, codes=P, scales=P, saved=P, saved_scales=P)
    check(lib.moe_swiglu_save_e4m3, good, [
        (dict(R=-1), INV), (dict(f=0), UNS), (dict(f=24), UNS), (dict(ld=120), INV), (dict(ld=130), INV),
        (dict(codes=None), INV), (dict(scales=None), INV), (dict(g=None), INV), (dict(u=None), INV),
        (dict(saved=None), INV), (dict(saved_scales=None), INV), (dict(u=ODD), INV), (dict(h=ODD), INV),
        (dict(R=0, g=None, u=None), OK)])


def test_swiglu_backward(lib):
    good = dict(R=4, f=128, saved=P, saved_scales=P, dh=P, dg=P, du=P, ld=128, h=P, codes=P, scales=P)
    check(lib.moe_swiglu_backward_e4m3, good, [
        (dict(R=-1), INV), (dict(f=8), UNS), (dict(f=144, ld=144), UNS), (dict(ld=64), INV), (dict(codes=None), INV),
        (dict(scales=None), INV), (dict(dh=None), INV), (dict(dg=None), INV), (dict(du=None), INV), (dict(saved=None), INV),
        (dict(dg=ODD), INV), (dict(R=0, dh=None), OK)])


def test_wgrad(lib):
    good = dict(R=4, N=128, K=256, E=2, x_dtype=1, dw_dtype=0, acc=0, dy=P, ld=128, x=P, sx=None, off=P, dw=P)
    check(lib.moe_grouped_wgrad, good, [
        (dict(R=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(E=0), INV), (dict(N=120), UNS), (dict(K=8), UNS),
        (dict(E=2000), UNS), (dict(x_dtype=0), UNS), (dict(dw_dtype=3), UNS), (dict(ld=64), INV), (dict(ld=132), INV),
        (dict(sx=P), INV), (dict(x_dtype=2), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(off=None), INV),
        (dict(dw=None), INV), (dict(dy=ODD), INV), (dict(dw=ODD), INV), (dict(R=0, acc=1, dy=None, x=None), OK)])


def test_router_losses(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_router_losses_workspace_size_for(4096, 256, 152, ctypes.byref(n)) == OK and n.value > 0
    assert lib.moe_router_losses_workspace_size_for(4096, 256, 0, ctypes.byref(n)) == INV
    assert lib.moe_router_losses_workspace_size_for(4096, 2000, 152, ctypes.byref(n)) == UNS
    assert lib.moe_router_losses_workspace_size_for(4096, 256, 152, None) == INV
    good = dict(T=4, E=8, k=2, logits=P, idx=P, mask=None, b=0.1, z=0.1, loss=P, counts=P, lse=P, ws=P, size=1 << 20)
    check(lib.moe_router_losses, good, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=9), INV), (dict(E=1025), UNS),
        (dict(E=64, k=33), UNS), (dict(logits=None), INV), (dict(idx=None), INV), (dict(loss=None), INV),
        (dict(counts=None), INV), (dict(lse=None), INV), (dict(logits=ODD), INV)])
    good = dict(T=4, E=8, k=2, logits=P, idx=P, mask=None, b=0.1, z=0.1, counts=P, lse=P, grad=None, w=P, dw=P, out=P)
    check(lib.moe_router_losses_backward, good, [
        (dict(T=-1), INV), (dict(k=9), INV), (dict(w=None), INV), (dict(dw=None), INV), (dict(idx=None), INV),
        (dict(logits=None), INV), (dict(counts=None), INV), (dict(lse=None), INV), (dict(out=None), INV),
        (dict(out=ODD), INV), (dict(T=0, logits=None, out=None), OK)])


# ---- the binding: correctly sized CPU tensors stop at the device check

def b16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(*s)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


GEMM = dict(a=u8(6, 144), a_scales=f32(6, 2), offsets=i32(3), w=u8(2, 272, 144), w_scales=f32(2, 3, 2))
WGRAD = dict(dy=b16(6, 144), x=u8(6, 272), x_scales=f32(6, 3), offsets=i32(3))
SAVED = dict(saved=u8(2, 6, 144), saved_scales=f32(2, 6, 2), dh=b16(6, 144))


@pytest.mark.parametrize("fn,good", [
    (api.grouped_block_gemm, GEMM), (api.grouped_wgrad, WGRAD), (api.swiglu_backward, SAVED),
    (api.quantize_blocks, dict(x=b16(6, 144))), (api.swiglu_save, dict(g=b16(6, 144), u=b16(6, 144))),
    (api.router_losses, dict(logits=f32(6, 8), topk_idx=i32(6, 2), balance=1.0, z=1.0, workspace=u8(64)))])
def test_binding_refuses_other_sizes_and_types(fn, good):
    with pytest.raises(ValueError, match="device tensors"):
        fn(**good)
    for name, t in good.items():
        if not isinstance(t, torch.Tensor) or name == "workspace":
            continue
        if len(good) > 1:
            with pytest.raises(ValueError):
                fn(**dict(good, **{name: t[:-1]}))
        with pytest.raises(ValueError):
            fn(**dict(good, **{name: t.double()}))


def test_binding_refuses_other_arguments():
    with pytest.raises(ValueError, match="scale"):
        api.quantize_blocks(b16(2, 128), "max")
    with pytest.raises(ValueError, match="adjacent"):
        api.swiglu_save(b16(128, 8).T, b16(128, 8).T)
    with pytest.raises(ValueError, match="pitch"):
        api.swiglu_save(b16(6, 256)[:, :128], b16(6, 128))
    with pytest.raises(ValueError, match="reduce"):
        api.grouped_block_gemm(**dict(GEMM, transposed=True))
    with pytest.raises(ValueError, match="out"):
        api.grouped_block_gemm(**GEMM, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="dw"):
        api.grouped_wgrad(**WGRAD, accumulate=True)
    with pytest.raises(ValueError, match="mask"):
        api.router_losses(f32(6, 8), i32(6, 2), 1.0, 1.0, mask=f32(6))
