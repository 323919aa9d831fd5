"""Trains one MoE FFN layer's experts and router in 8 bits: a layer learns to
imitate a fixed random function, with the library's operators from the router
to the weight gradients.

    python examples/train_experts.py [--steps 30] [--tokens 2048]

fp32 master weights are kept; after each step the experts are laid out again
as E4M3 codes with a scale for each 128 x 128 block (gate and up as one
matrix).  For the backward pass a step keeps the token rows, the gate and the
up activations in 8 bits and nothing else of the experts.  The elementwise
glue around the library's calls (the loss, the router's product) is plain
torch.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from routed_expert_ffn_gemm_gb300 import api  # noqa: E402

F8 = torch.float8_e4m3fn


def quantize_weights(w):
    """E4M3 codes [E, N, K] and scales [E, N/128, K/128] of fp32 weights whose
    sizes are multiples of 128."""
    E, N, K = w.shape
    b = w.view(E, N // 128, 128, K // 128, 128)
    s = (b.abs().amax((2, 4)) / 448).clamp_min(2.0 ** -100)
    q = (b / s[:, :, None, :, None]).clamp(-448, 448).to(F8)
    return q.reshape(E, N, K).view(torch.uint8), s


class Layer:
    def __init__(self, d, ffn, E, k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return std * torch.randn(*shape, generator=g, device=device)

        self.d, self.ffn, self.E, self.k = d, ffn, E, k
        self.w_router = normal(E, d, std=d ** -0.5).bfloat16()
        self.w_gu = normal(E, 2 * ffn, d, std=d ** -0.5)  # gate, then up
        self.w_down = normal(E, d, ffn, std=ffn ** -0.5)
        self.lay_out()

    def lay_out(self):
        """The experts' weights as the products take them."""
        self.q_gu, self.s_gu = quantize_weights(self.w_gu)
        self.q_down, self.s_down = quantize_weights(self.w_down)

    def forward(self, x, balance=1e-2, z=1e-3):
        """out [T, d] of x [T, d] bf16, and what backward() needs."""
        T, E, k, d, f = x.shape[0], self.E, self.k, self.d, self.ffn
        p = api.problem(T, d, f, E, k)
        new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=x.device)  # noqa: E731
        logits, idx, w = new(T, E, dtype=torch.float32), new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        api.moe_router_topk(p, x, self.w_router, None, None, logits, idx, w)
        moved = api.dispatch(x, idx, E)
        offsets, row = moved.offsets, moved.inv_row
        # powers of two: the same codes are the weight gradient's checkpoint
        x_codes, x_scales = api.quantize_blocks(moved.rows, "pow2")
        gu = api.grouped_block_gemm(x_codes, x_scales, offsets, self.q_gu, self.s_gu)
        h = api.swiglu_save(gu[:, :f], gu[:, f:])
        y = api.grouped_block_gemm(h.codes, h.scales, offsets, self.q_down, self.s_down)
        out = api.combine(y, row, w)
        losses = api.router_losses(logits, idx, balance, z)
        return out, losses, (p, x, logits, idx, w, offsets, row, x_codes, x_scales, h.saved, h.saved_scales, y)

    def backward(self, d_out, losses, kept):
        """Gradients of x, w_gu, w_down and w_router from d_out [T, d] bf16."""
        p, x, logits, idx, w, offsets, row, x_codes, x_scales, saved, saved_scales, y = kept
        dy, d_w = api.combine_backward(d_out, y, row, w)
        # the experts'
        dy_codes, dy_scales = api.quantize_blocks(dy, "amax")
        dh = api.grouped_block_gemm(dy_codes, dy_scales, offsets, self.q_down, self.s_down, transposed=True)
        g = api.swiglu_backward(saved, saved_scales, dh, want_h=True, want_codes=True)
        d_down = api.grouped_wgrad(dy, g.h, None, offsets)
        d_gu = api.grouped_wgrad(g.d_gu, x_codes, x_scales, offsets)
        dx_rows = api.grouped_block_gemm(g.codes, g.scales, offsets, self.q_gu, self.s_gu, transposed=True)
        dx = api.dispatch_backward(dx_rows, row)
        # the router's
        d_logits = api.router_losses_backward(logits, idx, losses, topk_w=w, d_topk_w=d_w)
        dx = (dx.float() + d_logits @ self.w_router.float()).bfloat16()
        return dx, d_gu, d_down, d_logits.T @ x.float()

    def step(self, x, target, rate):
        """One step of gradient descent on the mean squared error; returns the
        error and the router's losses before it."""
        out, losses, kept = self.forward(x)
        diff = out.float() - target.float()
        _, d_gu, d_down, d_router = self.backward((2 * diff / diff.shape[0]).bfloat16(), losses, kept)
        self.w_gu -= rate * d_gu
        self.w_down -= rate * d_down
        self.w_router = (self.w_router.float() - rate * d_router).bfloat16()
        self.lay_out()
        return (diff * diff).sum(1).mean(), losses.loss, losses.counts


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--rate", type=float, default=0.2)
    a = ap.parse_args(argv)
    d, ffn, E, k = 512, 768, 16, 4
    layer = Layer(d, ffn, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, d, generator=g, device="cuda").bfloat16()
    target = torch.tanh(x.float() @ (torch.randn(d, d, generator=g, device="cuda") * d ** -0.5)).bfloat16()
    errors = []
    for i in range(a.steps):
        error, loss, counts = layer.step(x, target, a.rate)
        errors.append(float(error))
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  error {errors[-1]:9.3f}  balance {float(loss[0]):.5f}  z {float(loss[1]):.5f}  "
                  f"rows of an expert {int(counts[:E].min())} to {int(counts[:E].max())}")
    status = api.moe_read_device_status()
    assert status == api.OK, api.moe_status_string(status)
    return errors


if __name__ == "__main__":
    main()
