"""The operators around a layer's routed experts in 4 bits, and the gradients of its token movement, as they are measured:

  dispatch   tokens sorted by expert (padding tokens and dropped assignments take no row), and the gradient of that
  combine    the experts' rows weighted and summed back to tokens, and the gradient of that
  quantize   MXFP4: blocks of 32 in E2M1 with a power of two each, quantised and read back
  gateup     tokens dispatched as MXFP4 rows, and the grouped 4-bit product on them
  down       SwiGLU to MXFP4 rows, and the grouped 4-bit product on them
  product    the grouped 4-bit product by itself

Rows are grouped by expert: rows offsets[e] to offsets[e + 1] belong to expert e; rows behind the last are left as they were."""
import math

import numpy as np
import torch

own = False
B = 32
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the codes 0 to 7; codes 8 to 15 are their negatives
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# hidden size, expert width, experts and experts a token of the layer shapes that this framework's workloads use
WIDE = {"d": 7168, "ffn": 2048, "E": 256, "k": 8}
NARROW = {"d": 2048, "ffn": 768, "E": 128, "k": 8}
FEW = {"d": 4096, "ffn": 14336, "E": 8, "k": 2}


def listed():
    return [
        # a decode batch's tokens sorted by expert: latency
        dict(name="dispatch-decode", op="dispatch", T=64, E=WIDE["E"], k=WIDE["k"], d=WIDE["d"], x="bf16", skew=0.6, drop=0.0, backward=False),
        # a training batch of packed sequences with padding tokens and some assignments past their expert's capacity
        dict(name="dispatch-train", op="dispatch", T=16384, E=NARROW["E"], k=NARROW["k"], d=NARROW["d"], x="bf16", skew=0.6, drop=0.07, backward=False),
        # the same batch's gradient of the tokens, added to what reaches them through the router
        dict(name="dispatch-gradient", op="dispatch", T=16384, E=NARROW["E"], k=NARROW["k"], d=NARROW["d"], x="bf16", skew=0.6, drop=0.07, backward=True),
        # a decode batch's experts back to tokens, with a shared expert's output: latency
        dict(name="combine-decode", op="combine", T=64, E=WIDE["E"], k=WIDE["k"], d=WIDE["d"], x="bf16", skew=0.6, drop=0.0, backward=False),
        # a training batch on few wide experts: gradients of the experts' rows and of the routing weights
        dict(name="combine-gradient", op="combine", T=16384, E=FEW["E"], k=FEW["k"], d=FEW["d"], x="bf16", skew=0.3, drop=0.0, backward=True),
        # the rows of a ragged prompt in fp32, scales that clip nothing
        dict(name="quantize-prompt", op="quantize", E=0, R=1049, C=NARROW["d"], x="f32", scale="fit"),
        # the master weights of a layer's shard after a step, laid out for the product and read back for the straight-through forward
        dict(name="quantize-weights", op="quantize", E=16, R=2 * WIDE["ffn"], C=WIDE["d"], x="bf16", scale="floor"),
        # one token decoded, gate and up as one product: 8 of 256 experts hold one row each. Latency and weight bytes count.
        dict(name="gateup-token", op="gateup", T=1, E=WIDE["E"], k=WIDE["k"], K=WIDE["d"], N=2 * WIDE["ffn"], skew=0.0, drop=0.0, scale="floor", out="bf16"),
        # a prompt's chunk over many experts, about a hundred rows each
        dict(name="gateup-prompt", op="gateup", T=4096, E=WIDE["E"], k=WIDE["k"], K=WIDE["d"], N=2 * WIDE["ffn"], skew=0.3, drop=0.0, scale="floor", out="bf16"),
        # a decode batch of 64 tokens through the down product: a few rows for each expert
        dict(name="down-batch", op="down", R=512, E=WIDE["E"], K=WIDE["ffn"], N=WIDE["d"], skew=0.6, scale="floor", out="bf16"),
        # a long prompt through narrow experts: rows in and out bound it
        dict(name="down-prompt", op="down", R=65536, E=NARROW["E"], K=NARROW["ffn"], N=NARROW["d"], skew=0.6, scale="fit", out="bf16"),
        # a long prompt on few wide experts: the product that the tensor cores bound
        dict(name="product-wide", op="product", R=16384, E=FEW["E"], K=FEW["d"], N=2 * FEW["ffn"], skew=0.3, scale="floor", out="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step, max(-(-lo // step), int(round(v / step)))) * step


def draw(rng):
    op = rng.choice(["dispatch", "combine", "quantize", "gateup", "down", "product"])
    skew, scale = rng.choice([0.0, 0.3, 0.6]), rng.choice(["floor", "fit"])
    if op in ("dispatch", "combine"):
        E = _spread(rng, 2, 512)
        k, d = rng.randint(1, min(8, E)), _spread(rng, 128, 8192, 8)
        T = max(1, min(_spread(rng, 1, 131072), (1 << 28) // (k * d)))
        return dict(op=op, T=T, E=E, k=k, d=d, x=rng.choice(["bf16", "bf16", "f32"]), skew=skew, drop=rng.choice([0.0, 0.1, 0.5]), backward=rng.random() < 0.5)
    if op == "quantize":
        E, C = rng.choice([0, 0, _spread(rng, 1, 64)]), _spread(rng, 128, 14336, 32)
        return dict(op=op, E=E, R=max(1, min(_spread(rng, 1, 65536), (1 << 28) // (C * max(1, E)))), C=C, x=rng.choice(["bf16", "bf16", "f32"]), scale=scale)
    E, K, N = _spread(rng, 2, 256), _spread(rng, 128, 7168, 32), _spread(rng, 128, 14336, 16)
    while E * N * K > 1 << 32:
        E = max(2, E // 2)
        N = N if E > 2 else N // 32 * 16
    R = _spread(rng, 1, 65536)
    while 2.0 * R * N * K > 1.9e12:
        R //= 2
    c = dict(op=op, E=E, K=K, N=N, skew=skew, scale=scale, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gateup":
        k = rng.randint(1, min(8, E))
        return dict(c, T=max(1, R // k), k=k, drop=rng.choice([0.0, 0.1]))
    return dict(c, R=R)


# ---------------------------------------------------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------------------------------------------------

def _dropped(c):
    """Padding tokens, and single assignments of the others, that take no row."""
    pad = int(c["drop"] * c["T"])
    return pad, ((c["T"] - pad) * c["k"] // 64 if c["drop"] else 0)


def _routes(c, g):
    """Distinct experts [T, k] of each token, popular ones more often; -1 where an assignment takes no row."""
    T, E, k = c["T"], c["E"], c["k"]
    bias = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
    score = bias[torch.randperm(E, generator=g, device="cuda")] - torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    pad, single = _dropped(c)
    order = torch.randperm(T, generator=g, device="cuda")
    rest = order[pad:].sort().values
    at = torch.randperm(rest.numel() * k, generator=g, device="cuda")[:single]
    idx[rest[at // k], at % k] = -1
    idx[order[:pad]] = -1
    return idx.contiguous()


def _counts(c):
    """Rows of each expert, largest first: shares rank^-skew."""
    share = np.arange(1, c["E"] + 1, dtype=np.float64) ** -c["skew"]
    want = share / share.sum() * c["R"]
    n = np.floor(want).astype(np.int64)
    n[np.argsort(n - want, kind="stable")[: c["R"] - n.sum()]] += 1
    return n


def _sorted(idx, E):
    """offsets [E + 1], counts [E], row_token [R], inv_row [T, k] of the assignments in expert order, earlier ones first."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    r = torch.arange(flat.numel(), device=idx.device)
    live = r < offsets[E]
    token = torch.where(live, order // idx.shape[1], torch.full_like(order, -1))
    inv = torch.empty_like(order)
    inv[order] = torch.where(live, r, torch.full_like(r, -1))
    return offsets.int(), counts.int(), token.int(), inv.int().view(idx.shape)


def _scale_exponents(a, kind):
    m, e = torch.frexp(a)
    p = e - 3 if kind == "floor" else torch.where(m <= 0.75, e - 3, e - 2)
    return torch.where(a > 0, p.clamp(-127, 127), torch.zeros_like(p))


def _mx(x, kind):
    """E2M1 values of the blocks of 32 of x, [..., C / 32, 32], and their exponents."""
    b = x.float().reshape(*x.shape[:-1], -1, B)
    p = _scale_exponents(b.abs().amax(-1), kind)
    q = torch.ldexp(b, -p[..., None])
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(q / step) * step).clamp(-6, 6), p


def _mx_values(x, kind):
    q, p = _mx(x, kind)
    return torch.ldexp(q, p[..., None]).reshape(x.shape)


def _packed(q):
    """Two codes a byte, the first in the low half."""
    a = q.abs().reshape(*q.shape[:-2], -1)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= (q.reshape(a.shape) < 0).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _weights(E, N, K, g):
    """Codes [E, N, K / 2] and scales [E, K / 32, N] of normal weights."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, K // B, N, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        q, p = _mx(torch.randn(min(step, E - e), N, K, generator=g, device="cuda") / math.sqrt(K), "floor")
        codes[e : e + step] = _packed(q)
        scales[e : e + step] = (p + 127).to(torch.uint8).transpose(1, 2)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, s = dict(case), {}

    def normal(*shape, dtype=torch.bfloat16):
        # activations: a normal body with a row's own magnitude
        x = torch.randn(*shape, generator=g, device="cuda")
        return (x * torch.exp(0.5 * torch.randn(shape[0], *(1,) * (len(shape) - 1), generator=g, device="cuda"))).to(dtype)

    if c["op"] in ("dispatch", "combine"):
        T, k, d, t = c["T"], c["k"], c["d"], DT[c["x"]]
        s["idx"] = _routes(c, g)
        s["inv"] = _sorted(s["idx"], c["E"])[3]
        if c["op"] == "combine":
            s["w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
            s["y"] = normal(T * k, d, dtype=t)
            if c["backward"]:
                s["dout"], s["dy"] = normal(T, d, dtype=t), torch.zeros(T * k, d, dtype=t, device="cuda")
            else:
                s["add"] = normal(T, d, dtype=t)
        elif c["backward"]:
            s["dr"], s["add"] = normal(T * k, d, dtype=t), normal(T, d, dtype=t)
        else:
            s["t"], s["rows"] = normal(T, d, dtype=t), torch.zeros(T * k, d, dtype=t, device="cuda")
    elif c["op"] == "quantize":
        s["t"] = normal(*((c["E"],) if c["E"] else ()), c["R"], c["C"], dtype=DT[c["x"]])
    else:
        E, K, N = c["E"], c["K"], c["N"]
        if c["op"] == "gateup":
            s["idx"], s["t"] = _routes(c, g), normal(c["T"], K)
            c["R"] = c["T"] * c["k"]
            s["cap"] = int(_sorted(s["idx"], E)[1].max())
        else:
            n = np.random.RandomState(seed & 0x7FFFFFFF).permutation(_counts(c))
            s["offsets"], s["cap"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda(), int(n.max())
            if c["op"] == "down":
                s["gu"] = normal(c["R"], 2 * K)
            else:
                q, p = _mx(normal(c["R"], K), c["scale"])
                s["a"], s["sa"] = _packed(q), (p + 127).to(torch.uint8)
        s["weights"], s["sw"] = _weights(E, N, K, g)
        s["y"] = torch.zeros(c["R"], N, dtype=DT[c["out"]], device="cuda")
    return {**c, **s}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def _kernels(s):
    from routed_expert_ffn_gemm_gb300 import api

    if s["op"] == "dispatch":
        if s["backward"]:
            return api.dispatch_backward(s["dr"], s["inv"], add=s["add"])
        r = api.dispatch(s["t"], s["idx"], s["E"], rows=s["rows"])
        return r.rows, r.offsets, r.counts, r.row_token, r.inv_row
    if s["op"] == "combine":
        if s["backward"]:
            r = api.combine_backward(s["dout"], s["y"], s["inv"], s["w"], dy=s["dy"])
            return r.dy, r.dw
        return api.combine(s["y"], s["inv"], s["w"], add=s["add"])
    if s["op"] == "quantize":
        codes, scales = api.quantize_mxfp4(s["t"], scale=s["scale"], weights=s["E"] > 0)
        return api.mxfp4_values(codes, scales, dtype=s["t"].dtype, weights=s["E"] > 0)
    if s["op"] == "gateup":
        r = api.dispatch(s["t"], s["idx"], s["E"], quantize=s["scale"])
        return api.grouped_mxfp4_gemm(r.rows, r.scales, r.offsets, s["weights"], s["sw"], out=s["y"]), r.inv_row
    if s["op"] == "down":
        f = s["K"]
        r = api.swiglu_mxfp4(s["gu"][:, :f], s["gu"][:, f:], scale=s["scale"])
        return api.grouped_mxfp4_gemm(r.codes, r.scales, s["offsets"], s["weights"], s["sw"], out=s["y"])
    return api.grouped_mxfp4_gemm(s["a"], s["sa"], s["offsets"], s["weights"], s["sw"], out=s["y"])


def _code_values(codes, scales):
    """fp32 values [..., K] of codes [..., K / 2] with scales [..., K / 32]."""
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), device="cuda")
    pairs = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)
    x = pairs[codes.int()].reshape(*codes.shape[:-1], -1, B)
    x *= torch.exp2(scales.float() - 127)[..., None]
    return x.reshape(*codes.shape[:-1], -1)


def _grouped(x, offsets, s):
    """Rows x [R, K] of fp32 values times their expert's weights: rows in one block of `cap` for each expert."""
    r = torch.arange(x.shape[0], device="cuda")
    live = r < offsets[-1]
    e = torch.bucketize(r, offsets[1:].long(), right=True).clamp_max(s["E"] - 1)
    at = torch.where(live, r - offsets.long()[e], torch.full_like(r, s["cap"]))
    blocks = torch.zeros(s["E"], s["cap"] + 1, x.shape[1], device="cuda")
    blocks[e, at] = x
    w = _code_values(s["weights"], s["sw"].transpose(1, 2))
    y = torch.bmm(blocks, w.transpose(1, 2))[e, at].to(s["y"].dtype)
    return torch.where(live[:, None], y, s["y"])


def _plain(s):
    if s["op"] == "dispatch":
        if s["backward"]:
            d = s["dr"][s["inv"].clamp_min(0).long()].float() * (s["inv"] >= 0)[..., None]
            return (s["add"].float() + d.sum(1)).to(s["add"].dtype)
        offsets, counts, token, inv = _sorted(s["idx"], s["E"])
        rows = torch.where((token >= 0)[:, None], s["t"][token.clamp_min(0).long()], s["rows"])
        return rows, offsets, counts, token, inv
    if s["op"] == "combine":
        there, at = s["inv"] >= 0, s["inv"].clamp_min(0).long()
        y = s["y"][at].float() * there[..., None]
        if not s["backward"]:
            return (s["add"].float() + (y * s["w"][..., None]).sum(1)).to(s["y"].dtype)
        d = s["dout"].float()[:, None]
        dy = (d * s["w"][..., None]).to(s["y"].dtype)
        # (rows that no assignment has keep what they hold; one row more takes what has none)
        out = torch.cat([s["dy"], s["dy"][:1]])
        out[torch.where(there, at, torch.full_like(at, s["y"].shape[0]))] = dy
        return out[:-1], (y * d).sum(2)
    if s["op"] == "quantize":
        return _mx_values(s["t"], s["scale"]).to(s["t"].dtype)
    if s["op"] == "gateup":
        offsets, _, token, inv = _sorted(s["idx"], s["E"])
        return _grouped(_mx_values(s["t"], s["scale"])[token.clamp_min(0).long()], offsets, s), inv
    if s["op"] == "down":
        g, u = s["gu"][:, : s["K"]].float(), s["gu"][:, s["K"] :].float()
        return _grouped(_mx_values(g * torch.sigmoid(g) * u, s["scale"]), s["offsets"], s)
    return _grouped(_code_values(s["a"], s["sa"]), s["offsets"], s)


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c, size = case, {"bf16": 2, "f32": 4}
    if c["op"] in ("dispatch", "combine"):
        pad, single = _dropped(c)
        R, n, d = c["T"] * c["k"], (c["T"] - pad) * c["k"] - single, c["d"]
        if c["op"] == "dispatch" and not c["backward"]:
            return {"bytes": size[c["x"]] * d * (c["T"] - pad + n) + 12 * R + 8 * c["E"], "flops": 0}
        if c["op"] == "dispatch" or not c["backward"]:
            weights = 4 * R if c["op"] == "combine" else 0
            return {"bytes": size[c["x"]] * d * (2 * c["T"] + n) + 4 * R + weights, "flops": 2.0 * n * d}
        return {"bytes": size[c["x"]] * d * (c["T"] + 2 * n) + 12 * R, "flops": 3.0 * n * d}
    if c["op"] == "quantize":
        n = max(1, c["E"]) * c["R"] * c["C"]
        # quantised (codes and scales written), then read back
        return {"bytes": 2 * n * size[c["x"]] + 2 * (n // 2 + n // B), "flops": 4.0 * n}
    K, N, R = c["K"], c["N"], c["R"] if "R" in c else c["T"] * c["k"]
    if c["op"] == "gateup":
        pad, single = _dropped(c)
        n = R - pad * c["k"] - single
        live = min(c["E"], n)
        extra = 2 * c["T"] * K + 12 * R + n * (K // 2 + K // B)  # tokens in, maps, and the quantised rows written
    else:
        n, live = R, int((_counts(c) > 0).sum())
        extra = (4 * R * K + R * (K // 2 + K // B) if c["op"] == "down" else 0) + 4 * c["E"]
    return {"bytes": extra + (n + live * N) * (K // 2 + K // B) + n * N * size[c["out"]], "flops": 2.0 * n * N * K}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _order64(idx, E):
    """Maps of the assignments by walking the experts."""
    i = idx.cpu().numpy()
    flat, k = i.reshape(-1), i.shape[1]
    groups = [np.flatnonzero(flat == e) for e in range(E)]
    row_of = np.concatenate(groups)
    token, inv = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    token[: row_of.size], inv[row_of] = row_of // k, np.arange(row_of.size)
    counts = np.array([len(x) for x in groups], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return [torch.from_numpy(x).cuda() for x in (offsets, counts, token, inv.reshape(i.shape))]


def _mx64(v, kind):
    """The values that MXFP4 keeps of v [..., C], in 64 bits."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[-1], B):
        b = v[..., c : c + B]
        top = b.abs().max(-1, keepdim=True).values
        p = torch.floor(torch.log2(top.clamp_min(1e-300)))
        p = torch.where(torch.exp2(p) > top, p - 1, p)
        p = torch.where(torch.exp2(p + 1) <= top, p + 1, p) - 2
        if kind == "fit":
            p = torch.where(top > 6 * torch.exp2(p), p + 1, p)
        p = torch.where(top > 0, p, torch.zeros_like(p))
        x = (b / torch.exp2(p)).abs()
        # the midpoints of neighbouring values; at a midpoint the even code is the lower one of every second pair
        q = torch.zeros_like(x)
        for i in range(7):
            mid = (VALUES[i] + VALUES[i + 1]) / 2
            q += (VALUES[i + 1] - VALUES[i]) * (x >= mid if i % 2 else x > mid).double()
        out[..., c : c + B] = torch.where(b < 0, -q, q) * torch.exp2(p)
    return out


def _wide(codes, scales):
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), dtype=torch.float64, device="cuda")
    x = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = v[(codes & 15).long()], v[(codes >> 4).long()]
    return x * torch.exp2(scales.double() - 127).repeat_interleave(B, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("dispatch", "combine"):
        n, inv = s["T"] * s["k"], s["inv"].long()
        if s["op"] == "dispatch" and not s["backward"]:
            offsets, counts, token, inv = _order64(s["idx"], s["E"])
            rows, live = s["rows"].double(), int(offsets[-1])
            rows[:live] = s["t"].double()[token[:live].long()]
            return rows, offsets, counts, token, inv
        if not s["backward"] or s["op"] == "dispatch":
            total, y = s["add"].double(), s["y" if s["op"] == "combine" else "dr"]
            for j in range(s["k"]):
                at = torch.nonzero(inv[:, j] >= 0)[:, 0]
                part = y[inv[at, j]].double()
                total[at] += part * s["w"][at, j, None].double() if s["op"] == "combine" else part
            return total
        dy, dw = s["dy"].double(), torch.zeros(s["T"], s["k"], dtype=torch.float64, device="cuda")
        for j in range(s["k"]):
            at = torch.nonzero(inv[:, j] >= 0)[:, 0]
            d = s["dout"][at].double()
            dy[inv[at, j]] = d * s["w"][at, j, None].double()
            dw[at, j] = (s["y"][inv[at, j]].double() * d).sum(1)
        return dy, dw
    if s["op"] == "quantize":
        return _mx64(s["t"].double(), s["scale"])
    if s["op"] == "gateup":
        offsets, _, token, inv = _order64(s["idx"], s["E"])
        a = _mx64(s["t"].double(), s["scale"])[token.clamp_min(0).long()]
    else:
        offsets = s["offsets"]
        if s["op"] == "down":
            gu, f = s["gu"].double(), s["K"]
            a = _mx64(gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:], s["scale"])
        else:
            a = _wide(s["a"], s["sa"])
    y, off = s["y"].double(), offsets.tolist()
    for e in range(s["E"]):
        if off[e + 1] > off[e]:
            y[off[e] : off[e + 1]] = a[off[e] : off[e + 1]] @ _wide(s["weights"][e], s["sw"][e].T).T
    return (y, inv) if s["op"] == "gateup" else y
