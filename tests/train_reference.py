"""Plain 64-bit forms of the expert-training operators, for the tests: loops
over experts and blocks, on the CPU, from the definitions in include/moe.h."""

import torch

BLOCK = 128
F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // BLOCK)


def e4m3(codes):
    return codes.view(F8).to(torch.float32).double()


def widen(codes, scales):
    """code * scale of rows [..., C] with scales [..., blocks] in 64 bits."""
    s = scales.double().repeat_interleave(BLOCK, -1)[..., : codes.shape[-1]]
    return e4m3(codes) * s


def widen_matrix(codes, scales):
    s = scales.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    return e4m3(codes) * s[: codes.shape[0], : codes.shape[1]]


def quantize(x, kind):
    """Codes and scales bit for bit (every step an exact or correctly rounded
    fp32 operation)."""
    x = x.float()
    C = x.shape[-1]
    codes = torch.empty(x.shape, dtype=torch.uint8)
    scales = torch.empty(*x.shape[:-1], blocks(C))
    for b in range(blocks(C)):
        v = x[..., b * BLOCK: (b + 1) * BLOCK]
        fin = torch.isfinite(v)
        a = torch.where(fin, v.abs(), torch.zeros_like(v)).amax(-1)
        zero, a = a == 0, a.clamp_min(2.0 ** -100)
        if kind == "amax":
            s, t = a / torch.tensor(448.0), torch.tensor(448.0) / a
        else:
            m, e = torch.frexp(a)
            p = torch.where(m <= 0.875, e - 9, e - 8)
            s, t = torch.ldexp(torch.ones_like(a), p), torch.ldexp(torch.ones_like(a), -p)
        s, t = torch.where(zero, torch.ones_like(s), s), torch.where(zero, torch.ones_like(t), t)
        y = (torch.where(fin, v, torch.zeros_like(v)) * t[..., None]).clamp(-448.0, 448.0)
        c = y.to(F8).view(torch.uint8)
        codes[..., b * BLOCK: (b + 1) * BLOCK] = torch.where(fin, c, torch.full_like(c, 0x7F))
        scales[..., b] = s
    return codes, scales


def groups(offsets):
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def block_gemm(a, a_scales, offsets, w, w_scales, transposed):
    """(result, sum of the terms' magnitudes), both [R, N] in 64 bits; rows
    outside every group are NaN."""
    N = w.shape[2] if transposed else w.shape[1]
    y = torch.full((a.shape[0], N), float("nan"), dtype=torch.float64)
    mag = y.clone()
    x = widen(a, a_scales)
    for e, lo, hi in groups(offsets):
        if hi > lo:
            m = widen_matrix(w[e], w_scales[e])
            m = m if transposed else m.T
            y[lo:hi], mag[lo:hi] = x[lo:hi] @ m, x[lo:hi].abs() @ m.abs()
    return y, mag


def wgrad(dy, x, offsets):
    E = offsets.numel() - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = dw.clone()
    for e, lo, hi in groups(offsets):
        if hi > lo:
            dw[e] = dy[lo:hi].double().T @ x[lo:hi].double()
            mag[e] = dy[lo:hi].double().abs().T @ x[lo:hi].double().abs()
    return dw, mag


def silu_mul(g, u):
    return g / (1 + torch.exp(-g)) * u


def router(logits, idx, mask, balance, z):
    """Both losses as functions of the logits (64 bits, differentiable), and
    the counts with the token count behind them."""
    T, E = logits.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    n, k = int(live.sum()), idx.shape[1]
    counts = torch.bincount(idx[live].reshape(-1).long(), minlength=E)
    out = torch.cat([counts, torch.tensor([n])]).to(torch.int32)
    if n == 0:
        return logits.sum() * 0, logits.sum() * 0, out
    p = torch.softmax(logits[live], 1)
    lse = torch.logsumexp(logits[live], 1)
    f = counts.double() / (n * k)
    return balance * E * (f * p.mean(0)).sum(), z * (lse * lse).mean(), out
