"""Plain forms of the 4-bit operators and the token movement, for the tests: on
the CPU, in 64 bits or bit for bit, from the definitions in include/moe.h."""

import torch

from tests.train_reference import groups

BLOCK = 32
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def unpack(codes):
    """uint8 [..., C / 2] to code numbers [..., C], the low half first."""
    return torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def widen(codes, scales):
    """The values of codes [..., C / 2] with scales [..., C / 32] in 64 bits."""
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return E2M1[unpack(codes).long()] * s.repeat_interleave(BLOCK, -1)


def quantize(x, kind):
    """Codes [..., C / 2] and scales [..., C / 32] bit for bit, by looking for
    the nearest of the eight magnitudes."""
    v = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    a = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    p = torch.full_like(a, -127)
    for i in range(-127, 128):  # the largest power with 4 * 2^i <= a, or the least with 6 * 2^i >= a
        at = torch.tensor(2.0, dtype=torch.float64) ** i
        if kind == "floor":
            p = torch.where(a >= 4 * at, torch.full_like(p, i), p)
        else:
            p = torch.where(a > 6 * at, torch.full_like(p, i + 1), p)
    p = torch.where(a == 0, torch.zeros_like(p), p)
    y = v / torch.exp2(p)[..., None]
    y = torch.where(bad[..., None], torch.zeros_like(y), y)
    gap = (y.abs()[..., None] - E2M1[:8]).abs()
    near = gap.amin(-1, keepdim=True)
    is_near = gap == near
    even = torch.tensor([c % 2 == 0 for c in range(8)])
    best = torch.where((is_near & even).any(-1), (is_near & even).int().argmax(-1), is_near.int().argmax(-1))
    code = (best + 8 * torch.signbit(y).long()).to(torch.uint8).reshape(x.shape)
    scales = torch.where(bad, torch.full_like(p, 255), p + 127).to(torch.uint8)
    return pack(code), scales


def product(a, a_scales, offsets, w, w_scales):
    """(result, sum of the terms' magnitudes), both [R, N] in 64 bits; rows
    outside every group are NaN."""
    y = torch.full((a.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    mag = y.clone()
    x = widen(a, a_scales)
    for e, lo, hi in groups(offsets):
        if hi > lo:
            m = widen(w[e], w_scales[e].T.contiguous()).T
            y[lo:hi], mag[lo:hi] = x[lo:hi] @ m, x[lo:hi].abs() @ m.abs()
    return y, mag


def maps(idx, E):
    """offsets, counts, row_token, inv_row by walking the experts."""
    flat, k = idx.reshape(-1), idx.shape[1]
    mine = [torch.nonzero(flat == e)[:, 0] for e in range(E)]
    counts = torch.tensor([m.numel() for m in mine], dtype=torch.int32)
    order = torch.cat(mine)
    inv = torch.full((flat.numel(),), -1, dtype=torch.int32)
    inv[order] = torch.arange(order.numel(), dtype=torch.int32)
    token = torch.full((flat.numel(),), -1, dtype=torch.int32)
    token[: order.numel()] = (order // k).to(torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    return offsets, counts, token, inv.view(idx.shape)


def combine(y, inv, w=None, add=None):
    """(result, sum of the terms' magnitudes) in 64 bits."""
    T, k = inv.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64) if add is None else add.double().clone()
    mag = out.abs()
    for j in range(k):
        on = inv[:, j] >= 0
        term = y[inv[on, j].long()].double() * (1 if w is None else w[on, j, None].double())
        out[on] += term
        mag[on] += term.abs()
    return out, mag


def combine_backward(d_out, y, inv, w):
    """dy (rows that no assignment has: NaN), dw and the magnitudes of dw's terms."""
    dy = torch.full(y.shape, float("nan"), dtype=torch.float64)
    dw = torch.zeros(inv.shape, dtype=torch.float64)
    mag = dw.clone()
    for j in range(inv.shape[1]):
        on = inv[:, j] >= 0
        r, d = inv[on, j].long(), d_out[on].double()
        dy[r] = d * (1 if w is None else w[on, j, None].double())
        terms = d * y[r].double()
        dw[on, j], mag[on, j] = terms.sum(1), terms.abs().sum(1)
    return dy, dw, mag
