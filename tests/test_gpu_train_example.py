"""examples/train_experts.py: its gradients against automatic differentiation
of the same layer in fp32, and that training lowers the error."""

import importlib.util
import os

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    build.build()
    spec = importlib.util.spec_from_file_location("train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def widen(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1).repeat_interleave(128, 2)


@pytest.mark.parametrize("T,d,ffn,E,k", [(37, 256, 128, 4, 2), (300, 384, 256, 8, 3)])
def test_gradients_of_a_step(example, T, d, ffn, E, k):
    layer = example.Layer(d, ffn, E, k, seed=T)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    d_out = (torch.randn(T, d, generator=g, device="cuda") / T).bfloat16()
    out, losses, kept = layer.forward(x, balance=0.3, z=0.02)
    got = layer.backward(d_out, losses, kept)
    idx = kept[3].long()

    x32, wr = x.float().requires_grad_(), layer.w_router.float().requires_grad_()
    w_gu = widen(layer.q_gu, layer.s_gu).requires_grad_()
    w_down = widen(layer.q_down, layer.s_down).requires_grad_()
    logits = x32 @ wr.T
    w = torch.softmax(logits.gather(1, idx), 1)
    want = 0
    for j in range(k):
        gu = torch.einsum("td,tnd->tn", x32, w_gu[idx[:, j]])
        h = torch.nn.functional.silu(gu[:, :ffn]) * gu[:, ffn:]
        want = want + w[:, j, None] * torch.einsum("tf,tdf->td", h, w_down[idx[:, j]])
    f = torch.bincount(idx.reshape(-1), minlength=E).float() / (T * k)
    p = torch.softmax(logits, 1)
    loss = 0.3 * E * (f * p.mean(0)).sum() + 0.02 * (torch.logsumexp(logits, 1) ** 2).mean()
    ((want * d_out.float()).sum() + loss).backward()
    # each 8-bit rounding (rows twice forward, once or twice backward, the
    # checkpoint) is 2^-4 at most and 2^-4 / sqrt(12) = 1.8 % rms of an
    # element; a handful of independent ones stay under 10 % of the norm
    for a, b in ((out, want.detach()), (got[0], x32.grad), (got[1], w_gu.grad), (got[2], w_down.grad), (got[3], wr.grad)):
        assert (a.float() - b).norm() <= 0.1 * b.norm()
    assert api.moe_read_device_status() == api.OK


def test_training_lowers_the_error(example):
    errors = example.main(["--steps", "30", "--tokens", "1024"])
    assert errors[-1] < 0.7 * errors[0]
