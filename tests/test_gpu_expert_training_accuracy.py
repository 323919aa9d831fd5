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
