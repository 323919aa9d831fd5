"""Accuracy of the expert-training operators where their fp32 arithmetic is
stretched: logits of large magnitude, gates far below zero."""

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests import train_reference as ref
from tests.test_gpu_expert_training import close, gen, routed

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


@pytest.mark.parametrize("balance,z", [(0.3, 0.0), (0.0, 0.02)], ids=["balance", "z"])
@pytest.mark.parametrize("shift", [0.0, 512.0, -8192.0, 65536.0])
@pytest.mark.parametrize("T,E,k", [(33, 8, 2), (40, 60, 4), (50, 256, 8)])
def test_router_gradient_of_shifted_logits(T, E, k, shift, balance, z):
    # A constant added to a row's logits changes none of its probabilities.
    # The logits are multiples of 2^-7, so that adding it is exact; lse, of
    # the constant's magnitude, is rounded to fp32 and with it off by up to
    # 2^-9, and may not carry that into the probabilities.
    logits, idx, _ = routed(T, E, k, seed=T)
    logits = torch.round(logits * 128) / 128 + shift
    l64 = logits.double().requires_grad_()
    lb, lz, _ = ref.router(l64, idx, None, balance, z)
    (lb + lz).backward()
    logits, idx = logits.to(DEV), idx.to(DEV)
    r = api.router_losses(logits, idx, balance, z)
    close(r.loss, torch.stack([lb, lz]).detach())
    close(api.router_losses_backward(logits, idx, r), l64.grad)


def gates(lo=-65.0, hi=20.0, rows=256):
    """Rows of 128 equal gates, bf16 values from lo to hi."""
    g = torch.linspace(lo, hi, rows).bfloat16()
    return g[:, None].expand(rows, 128).contiguous()


# an fp32 operation is off by half a unit of 2^-23 at most, expf and the
# approximate reciprocal by two and one, as CUDA's tables state

def test_swiglu_scales_follow_the_gate():
    # sigmoid 2 + 0.5 + 1, two products 0.5 each, the division by 448 0.5
    g = gates()
    r = api.swiglu_save(g.to(DEV), torch.ones_like(g).to(DEV))
    want = (g[:, :1].double() * torch.sigmoid(g[:, :1].double())).abs() / 448
    assert ((r.scales.cpu().double() - want).abs() <= 6 * 2.0 ** -23 * want)[want > 0].all()


def test_swiglu_gradient_scales_follow_the_gate():
    # du: as above.  dg: the sigmoid's 3.5; 1 + g (1 - s) 0.5 three times, at
    # most doubled where the addition cancels (|g| >= 2); three products and
    # the division
    g = gates(-60.0, -2.0)
    saved, scales = ref.quantize(torch.stack([g, torch.ones_like(g)]), "pow2")
    r = api.swiglu_backward(saved.to(DEV), scales.to(DEV), torch.ones_like(g).to(DEV), want_codes=True)
    v = ref.widen(saved, scales)[0, :, :1]
    s = torch.sigmoid(v)
    want = torch.cat([s * (1 + v * (1 - s)), v * s], 1).abs() / 448
    assert ((r.scales.cpu().double() - want).abs() <= torch.tensor([9.0, 6.0]) * 2.0 ** -23 * want).all()


def test_swiglu_of_infinite_and_nan_gates():
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([inf, -inf, nan, 3e38, -3e38, 0.0, -0.0, 1.0] * 16).bfloat16()[None]
    r = api.swiglu_save(g.to(DEV), torch.ones_like(g).to(DEV), want_h=True)
    want = ref.silu_mul(g.double(), torch.ones_like(g).double()).bfloat16()
    got = r.h.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert ((got == want) | torch.isnan(want) | ((got - want).abs() <= 2.0 ** -8 * want.abs())).all()
