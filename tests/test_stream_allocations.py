"""What a call with stream= makes for itself belongs to that stream: without a
GPU, with stand-ins that record which stream is current at each allocation,
copy and launch."""

import contextlib

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api


class Side:
    cuda_stream = 0x77


class Other:
    cuda_stream = 0x11


class Recorder:
    def __init__(self, monkeypatch):
        self.current, self.made, self.launched, self.kept = None, [], [], []
        side_of = {}

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        def made(fn):
            def call(*args, **kw):
                self.made.append((fn.__name__, self.current))
                return fn(*args, **kw)
            return call

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current or Other())
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: side_of.setdefault(h, SIDE))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.kept.append(t))
        monkeypatch.setattr(api, "_stream", lambda s: self.current if s is None else s)
        monkeypatch.setattr(api, "_ptr", lambda t: None if t is None else 0x1000)
        monkeypatch.setattr(api, "_pitched", lambda t: 0x1000)
        monkeypatch.setattr(api, "_call", lambda name, *args: self.launched.append((name, args[-1])))
        for name in ("empty", "empty_like"):
            monkeypatch.setattr(torch, name, made(getattr(torch, name)))
        reshape = torch.Tensor.reshape
        monkeypatch.setattr(torch.Tensor, "reshape", made(reshape))


SIDE = Side()


def b16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def check(monkeypatch, fn, args):
    r = Recorder(monkeypatch)
    out = fn(*args, stream=SIDE)
    assert r.made and r.launched, "nothing was recorded"
    assert all(s is SIDE for _, s in r.made), [n for n, s in r.made if s is not SIDE]
    assert all(s is SIDE for _, s in r.launched)
    tensors = [t for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)]
    assert tensors and all(any(t is k for k in r.kept) for t in tensors)


@pytest.mark.parametrize("x", [b16(6, 128), b16(3, 2, 128).transpose(0, 1), b16(128)], ids=["matrix", "copied", "row"])
def test_quantize_blocks(monkeypatch, x):
    check(monkeypatch, api.quantize_blocks, (x,))


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


f32 = torch.zeros
LOSSES = api.RouterLosses(f32(2), i32(9), f32(6), 1.0, 1.0)


@pytest.mark.parametrize("fn,args", [
    (api.grouped_block_gemm, (u8(6, 144), f32(6, 2), i32(3), u8(2, 272, 144), f32(2, 3, 2))),
    (api.swiglu_save, (b16(6, 144), b16(6, 144), True)),
    (api.swiglu_backward, (u8(2, 6, 128), f32(2, 6, 1), b16(6, 128), True, True)),
    (api.grouped_wgrad, (b16(6, 144), u8(6, 272), f32(6, 3), i32(3))),
    (api.router_losses, (f32(6, 8), i32(6, 2), 1.0, 1.0)),
    (api.router_losses_backward, (f32(6, 8), i32(6, 2), LOSSES))])
def test_training_operators(monkeypatch, fn, args):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(api, "_router_workspace", lambda *a: 64)
    check(monkeypatch, fn, args)


@pytest.mark.parametrize("want_routing", [False, True])
def test_layer_forward(monkeypatch, want_routing):
    monkeypatch.setattr(api, "moe_workspace_size", lambda p: 64)
    monkeypatch.setattr(api, "_check_layer", lambda *a: None)
    p = api.problem(6, 128, 128, 4, 2)
    names = ("w_router", "router_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down", "w_shared_gate",
             "w_shared_up", "w_shared_down")
    case = dict({n: None for n in names}, x=b16(6, 128))
    check(monkeypatch, api.layer_forward, (p, case, None, None, want_routing))
