"""The operators that train a layer's routed experts in 8 bits, as they are measured:

  quantize   rows to E4M3 with a scale for each block of 128 columns
  gemm       the grouped product of such rows with weights that have a scale for each 128 x 128 block, and its data gradient
  swiglu     SwiGLU that keeps its inputs in 8 bits, and its backward pass from them
  wgrad      the weight gradient of the grouped product, from 8-bit or bf16 activations
  router     the router's balance and z losses with the per-expert counts, and the gradient of the logits

Rows are grouped by expert: rows offsets[e] to offsets[e + 1] belong to expert e."""
import math

import numpy as np
import torch

own = False
B = 128
TOP = 448.0

# hidden size, expert width and experts of the layer shapes that this framework's workloads use
WIDE = {"d": 7168, "ffn": 2048, "E": 256}
NARROW = {"d": 2048, "ffn": 768, "E": 128}
FEW = {"d": 4096, "ffn": 14336, "E": 8}


def listed():
    return [
        # one token decoded: 8 of 256 experts hold one row each; gate and up as one product. Latency and weight bytes count.
        dict(name="gemm-one-token", op="gemm", E=WIDE["E"], R=8, K=WIDE["d"], N=2 * WIDE["ffn"], skew=0.0, empty=0.0, transposed=False, out="bf16"),
        # a decode batch of 64 tokens, the down product: a few rows for each expert, some experts without any
        dict(name="gemm-batch", op="gemm", E=WIDE["E"], R=512, K=WIDE["ffn"], N=WIDE["d"], skew=0.6, empty=0.1, transposed=False, out="bf16"),
        # a training or prefill batch on few wide experts: the product that the tensor cores bound
        dict(name="gemm-prefill", op="gemm", E=FEW["E"], R=16384, K=FEW["d"], N=2 * FEW["ffn"], skew=0.3, empty=0.0, transposed=False, out="bf16"),
        # the data gradient of gate and up through the forward's own weights, under skewed expert loads
        dict(name="gemm-data-gradient", op="gemm", E=NARROW["E"], R=65536, K=2 * NARROW["ffn"], N=NARROW["d"], skew=0.6, empty=0.0, transposed=True, out="bf16"),
        # the tokens of a decode batch before their product
        dict(name="quantize-decode", op="quantize", R=64, C=WIDE["d"], x="bf16", scale="amax"),
        # a training batch kept for the backward pass: scales are powers of two
        dict(name="quantize-train", op="quantize", R=65536, C=NARROW["d"], x="bf16", scale="pow2"),
        # a short ragged prompt, forward
        dict(name="swiglu-prompt", op="swiglu", R=1048, f=NARROW["ffn"], backward=False, coded=True),
        # a training batch, backward: gradients in bf16 for the weight gradient and in codes for the data gradient
        dict(name="swiglu-backward", op="swiglu", R=32768, f=WIDE["ffn"], backward=True, coded=True),
        # many experts with about a hundred rows each: the written gradients bound it
        dict(name="wgrad-many", op="wgrad", E=NARROW["E"], R=16384, N=2 * NARROW["ffn"], K=NARROW["d"], skew=0.6, empty=0.1, x="e4m3", out="f32"),
        # few wide experts, the down product's gradient from bf16 rows: the tensor cores bound it
        dict(name="wgrad-few", op="wgrad", E=FEW["E"], R=8192, N=FEW["d"], K=FEW["ffn"], skew=0.3, empty=0.0, x="bf16", out="bf16"),
        # a small layer's router: launches count
        dict(name="router-small", op="router", T=64, E=8, k=2, masked=0.0, weights=False),
        # a training batch with padding tokens and the gradient of the kept weights
        dict(name="router-train", op="router", T=32768, E=WIDE["E"], k=8, masked=0.07, weights=True),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step, max(-(-lo // step), int(round(v / step)))) * step


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quantize", "swiglu", "wgrad", "router"])
    load = dict(skew=rng.choice([0.0, 0.3, 0.6]), empty=rng.choice([0.0, 0.1, 0.5]))
    if op == "gemm":
        E, R = _spread(rng, 1, 256), _spread(rng, 1, 65536)
        K, N = _spread(rng, 128, 7168, 16), _spread(rng, 128, 28672, 16)
        while E * N * K > 1 << 33:
            E = max(1, E // 2)
        while 2.0 * R * N * K > 3.8e12:
            R //= 2
        return dict(op=op, E=E, R=R, K=K, N=N, transposed=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "f32"]), **load)
    if op == "wgrad":
        E, R = _spread(rng, 1, 256), _spread(rng, 1, 65536)
        N, K = _spread(rng, 128, 8192, 16), _spread(rng, 128, 14336, 16)
        while E * N * K > 470_000_000:
            E, N = (E // 2, N) if E > 1 else (E, max(128, N // 32 * 16))
        while 2.0 * R * N * K > 1.9e12:
            R //= 2
        return dict(op=op, E=E, R=R, N=N, K=K, x=rng.choice(["e4m3", "e4m3", "bf16"]), out=rng.choice(["f32", "bf16"]), **load)
    if op == "quantize":
        C = _spread(rng, 128, 14336, 16)
        return dict(op=op, R=min(_spread(rng, 1, 65536), (1 << 28) // C), C=C, x=rng.choice(["bf16", "bf16", "f32"]), scale=rng.choice(["amax", "pow2"]))
    if op == "swiglu":
        coded = rng.random() < 0.6
        f = _spread(rng, 128, 14336, 128 if coded else 16)
        return dict(op=op, R=min(_spread(rng, 1, 65536), (1 << 27) // f), f=f, backward=rng.random() < 0.5, coded=coded)
    E = _spread(rng, 2, 512)
    return dict(op=op, T=min(_spread(rng, 1, 131072), (1 << 24) // E), E=E, k=rng.randint(1, min(8, E)), masked=rng.choice([0.0, 0.1]), weights=rng.random() < 0.6)


# ---------------------------------------------------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------------------------------------------------

def _counts(case):
    """Rows of each expert, largest first: shares rank^-skew, `empty` of the experts without rows."""
    E, R = case["E"], case["R"]
    live = max(1, E - int(case["empty"] * E))
    share = np.arange(1, live + 1, dtype=np.float64) ** -case["skew"]
    want = share / share.sum() * R
    n = np.floor(want).astype(np.int64)
    n[np.argsort(n - want, kind="stable")[: R - n.sum()]] += 1
    return np.concatenate([n, np.zeros(E - live, np.int64)])


def _groups(case, seed):
    n = np.random.RandomState(seed & 0x7FFFFFFF).permutation(_counts(case))
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda(), int(n.max())


def _blocks(x, rows=False):
    """x [..., C] (or [..., N, C] for rows) as blocks of 128 (x 128), padded with zeros."""
    C = x.shape[-1]
    if rows:
        N = x.shape[-2]
        x = torch.nn.functional.pad(x, (0, -C % B, 0, -N % B))
        return x.reshape(*x.shape[:-2], x.shape[-2] // B, B, x.shape[-1] // B, B)
    return torch.nn.functional.pad(x, (0, -C % B)).reshape(*x.shape[:-1], -1, B)


def _row_codes(x, kind):
    """Plain E4M3 codes of rows (as float8) and the scale of each block of 128 columns."""
    b = _blocks(x.float())
    a = b.abs().amax(-1)
    if kind == "pow2":
        m, e = torch.frexp(a)
        s = torch.ldexp(torch.ones_like(a), torch.where(m <= TOP / 512, e - 9, e - 8))
    else:
        s = a / torch.full_like(a, TOP)
    s = torch.where(a > 0, s, torch.ones_like(s))
    q = (b / s[..., None]).clamp(-TOP, TOP).reshape(*b.shape[:-2], -1)[..., : x.shape[-1]]
    return q.contiguous().to(torch.float8_e4m3fn), s


def _weights(E, N, K, gen):
    """E4M3 codes [E, N, K] of normal weights with a scale for each 128 x 128 block."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-N // B), -(-K // B), device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        w = torch.randn(min(step, E - e), N, K, generator=gen, device="cuda") / math.sqrt(K)
        b = _blocks(w, rows=True)
        s = b.abs().amax((-3, -1)) / TOP
        s = torch.where(s > 0, s, torch.ones_like(s))
        q = (b / s[..., :, None, :, None]).clamp(-TOP, TOP).reshape(w.shape[0], b.shape[1] * B, b.shape[3] * B)[:, :N, :K]
        codes[e : e + step] = q.contiguous().to(torch.float8_e4m3fn).view(torch.uint8)
        scales[e : e + step] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, s = dict(case), {}

    def normal(*shape, dtype=torch.bfloat16):
        # activations: a normal body with a row's own magnitude
        x = torch.randn(*shape, generator=g, device="cuda")
        return (x * torch.exp(0.5 * torch.randn(shape[0], 1, generator=g, device="cuda"))).to(dtype)

    if c["op"] == "gemm":
        s["offsets"], s["cap"] = _groups(c, seed)
        q, s["a_scales"] = _row_codes(normal(c["R"], c["K"]), "amax")
        s["a"] = q.view(torch.uint8)
        s["w"], s["w_scales"] = _weights(c["E"], *((c["K"], c["N"]) if c["transposed"] else (c["N"], c["K"])), g)
    elif c["op"] == "wgrad":
        s["offsets"], s["cap"] = _groups(c, seed)
        s["dy"] = normal(c["R"], c["N"])
        s["x"], s["x_scales"] = normal(c["R"], c["K"]), None
        if c["x"] == "e4m3":
            q, s["x_scales"] = _row_codes(s["x"], "pow2")
            s["x"] = q.view(torch.uint8)
    elif c["op"] == "quantize":
        s["x"] = normal(c["R"], c["C"], dtype=torch.float32 if c["x"] == "f32" else torch.bfloat16)
    elif c["op"] == "swiglu":
        gu = normal(c["R"], 2 * c["f"])
        if c["backward"]:
            q, scales = _row_codes(torch.stack([gu[:, : c["f"]], gu[:, c["f"] :]]), "pow2")
            s["saved"], s["saved_scales"] = q.view(torch.uint8), scales.contiguous()
            s["dh"] = normal(c["R"], c["f"])
        else:
            s["gu"] = gu
    else:
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        top, idx = s["logits"].topk(k, dim=1)
        s["idx"], s["w"] = idx.to(torch.int32), torch.softmax(top, 1)
        s["dw"] = torch.randn(T, k, generator=g, device="cuda") / T if c["weights"] else None
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= c["masked"] if c["masked"] else None
        s["grad"] = torch.full((1,), 0.5, device="cuda")
        s["balance"], s["z"] = 1e-2, 1e-3
    return {**c, **s}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kernels(s):
    from routed_expert_ffn_gemm_gb300 import api

    if s["op"] == "gemm":
        return api.grouped_block_gemm(s["a"], s["a_scales"], s["offsets"], s["w"], s["w_scales"], transposed=s["transposed"], out_dtype=DT[s["out"]])
    if s["op"] == "wgrad":
        return api.grouped_wgrad(s["dy"], s["x"], s["x_scales"], s["offsets"], dw_dtype=DT[s["out"]])
    if s["op"] == "quantize":
        codes, scales = api.quantize_blocks(s["x"], scale=s["scale"])
        return codes.view(F8), scales
    if s["op"] == "swiglu":
        f = s["f"]
        if s["backward"]:
            r = api.swiglu_backward(s["saved"], s["saved_scales"], s["dh"], want_h=True, want_codes=s["coded"])
            return (r.d_gu, r.h) + ((r.codes.view(F8), r.scales) if s["coded"] else ())
        r = api.swiglu_save(s["gu"][:, :f], s["gu"][:, f:], want_h=not s["coded"], want_codes=s["coded"])
        return ((r.codes.view(F8), r.scales) if s["coded"] else (r.h,)) + (r.saved.view(F8), r.saved_scales)
    r = api.router_losses(s["logits"], s["idx"], s["balance"], s["z"], mask=s["mask"])
    dl = api.router_losses_backward(s["logits"], s["idx"], r, grad=s["grad"], topk_w=s["w"] if s["weights"] else None, d_topk_w=s["dw"], mask=s["mask"])
    return r.loss, r.counts, dl


def _padded(x, offsets, cap):
    """Rows in one block of `cap` for each expert, and where each row went."""
    r = torch.arange(x.shape[0], device="cuda")
    e = torch.bucketize(r, offsets[1:].long(), right=True)
    at = r - offsets.long()[e]
    out = torch.zeros(offsets.numel() - 1, cap, x.shape[1], device="cuda")
    out[e, at] = x
    return out, e, at


def _row_values(codes, scales):
    return codes.view(F8).float() * scales.repeat_interleave(B, -1)[..., : codes.shape[-1]]


def _plain(s):
    if s["op"] == "gemm":
        x, e, at = _padded(_row_values(s["a"], s["a_scales"]), s["offsets"], s["cap"])
        w = s["w"].view(F8).float()
        w *= s["w_scales"].repeat_interleave(B, 1)[:, : w.shape[1]].repeat_interleave(B, 2)[:, :, : w.shape[2]]
        return torch.bmm(x, w if s["transposed"] else w.transpose(1, 2))[e, at].to(DT[s["out"]])
    if s["op"] == "wgrad":
        x = s["x"].float() if s["x_scales"] is None else _row_values(s["x"], s["x_scales"])
        dy = _padded(s["dy"].float(), s["offsets"], s["cap"])[0]
        return torch.bmm(dy.transpose(1, 2), _padded(x, s["offsets"], s["cap"])[0]).to(DT[s["out"]])
    if s["op"] == "quantize":
        return _row_codes(s["x"], s["scale"])
    if s["op"] == "swiglu":
        f = s["f"]
        if s["backward"]:
            g, u = _row_values(s["saved"], s["saved_scales"]).unbind(0)
            dh, sig = s["dh"].float(), torch.sigmoid(g)
            d = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
            return (d.bfloat16(), (g * sig * u).bfloat16()) + (_row_codes(d, "amax") if s["coded"] else ())
        g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
        h = g * torch.sigmoid(g) * u
        return (_row_codes(h, "amax") if s["coded"] else (h.bfloat16(),)) + _row_codes(torch.stack([g, u]), "pow2")
    T, E, k = s["T"], s["E"], s["k"]
    live = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"].float()
    n = live.sum().clamp_min(1)
    p, lse = torch.softmax(s["logits"], 1), torch.logsumexp(s["logits"], 1)
    hot = torch.zeros(T, E, device="cuda").scatter_(1, s["idx"].long(), 1.0) * live[:, None]
    counts = hot.sum(0)
    f = counts / (n * k)
    loss = torch.stack([s["balance"] * E * (f * (p * live[:, None]).sum(0) / n).sum(), s["z"] * (lse * lse * live).sum() / n])
    d = s["balance"] * E * p * (f - (p * f).sum(1, keepdim=True)) + 2 * s["z"] * (lse[:, None] * p)
    d = d * (live[:, None] * s["grad"] / n)
    if s["weights"]:
        d = d.scatter_add(1, s["idx"].long(), s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True)))
    return loss, torch.cat([counts, live.sum()[None]]).to(torch.int32), d


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["op"] == "gemm":
        live = int((_counts(c) > 0).sum())
        R, N, K, kb, nb = c["R"], c["N"], c["K"], -(-c["K"] // B), -(-c["N"] // B)
        return {"bytes": R * K + 4 * R * kb + live * (N * K + 4 * nb * kb) + 4 * (c["E"] + 1) + R * N * size[c["out"]], "flops": 2.0 * R * N * K}
    if c["op"] == "wgrad":
        R, N, K = c["R"], c["N"], c["K"]
        scales = 4 * R * -(-K // B) if c["x"] == "e4m3" else 0
        return {"bytes": 2 * R * N + size[c["x"]] * R * K + scales + 4 * (c["E"] + 1) + c["E"] * N * K * size[c["out"]], "flops": 2.0 * R * N * K}
    if c["op"] == "quantize":
        n = c["R"] * c["C"]
        return {"bytes": n * (size[c["x"]] + 1) + 4 * c["R"] * -(-c["C"] // B), "flops": 4.0 * n}
    if c["op"] == "swiglu":
        n, s = c["R"] * c["f"], 4 * c["R"] * -(-c["f"] // B)
        if c["backward"]:
            return {"bytes": n * (4 + 6) + 2 * s + (2 * n + 2 * s if c["coded"] else 0), "flops": 16.0 * n}
        return {"bytes": n * (4 + 2) + 2 * s + (n + s if c["coded"] else 2 * n), "flops": 12.0 * n}
    T, E, k = c["T"], c["E"], c["k"]
    return {"bytes": 2 * 4 * T * E + 4 * T * k * (3 if c["weights"] else 1) + (T if c["masked"] else 0) + 4 * (E + 1) + 12, "flops": 12.0 * T * E}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _code64(v, pow2):
    """Codes (as the numbers they stand for) and scales of the last axis in blocks of 128, one block at a time."""
    codes, scales = torch.empty_like(v), []
    for c in range(0, v.shape[-1], B):
        b = v[..., c : c + B]
        top = b.abs().max(-1).values
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / TOP)))
            s = torch.where(top > s * TOP, 2 * s, s)
            s = torch.where(top <= s * (TOP / 2), s / 2, s)
        else:
            s = top / TOP
        s = torch.where(top > 0, s, torch.ones_like(s))
        x = b / s[..., None]
        # E4M3: steps of 2^(e - 3) for magnitudes in [2^e, 2^(e + 1)), e at least -6; torch.round goes to even
        step = torch.exp2(torch.frexp(x.abs())[1].clamp_min(-5).double() - 4)
        codes[..., c : c + B] = (torch.round(x / step) * step).clamp(-TOP, TOP)
        scales.append(s)
    return codes, torch.stack(scales, -1)


def _wide(codes, scales):
    out = codes.view(F8).double()
    for c in range(scales.shape[-1]):
        out[..., c * B : (c + 1) * B] *= scales[..., c, None].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("gemm", "wgrad"):
        off = s["offsets"].tolist()
        spans = [(e, off[e], off[e + 1]) for e in range(s["E"])]
    if s["op"] == "gemm":
        a = _wide(s["a"], s["a_scales"])
        y = torch.zeros(s["R"], s["N"], dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            if hi > lo:
                w = s["w"][e].view(F8).double()
                for i in range(s["w_scales"].shape[1]):
                    for j in range(s["w_scales"].shape[2]):
                        w[i * B : (i + 1) * B, j * B : (j + 1) * B] *= s["w_scales"][e, i, j].double()
                y[lo:hi] = a[lo:hi] @ (w if s["transposed"] else w.T)
        return y
    if s["op"] == "wgrad":
        x = s["x"].double() if s["x_scales"] is None else _wide(s["x"], s["x_scales"])
        dw = torch.zeros(s["E"], s["N"], s["K"], dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            dw[e] = s["dy"][lo:hi].double().T @ x[lo:hi]
        return dw
    if s["op"] == "quantize":
        return _code64(s["x"].double(), s["scale"] == "pow2")
    if s["op"] == "swiglu":
        f = s["f"]
        if s["backward"]:
            v = _wide(s["saved"], s["saved_scales"])
            g, u, dh = v[0], v[1], s["dh"].double()
            sig = 1 / (1 + torch.exp(-g))
            d = torch.cat([dh * u * (sig + g * sig * (1 - sig)), dh * (g * sig)], 1)
            return (d, g * sig * u) + (_code64(d, False) if s["coded"] else ())
        gu = s["gu"].double()
        h = gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:]
        return (_code64(h, False) if s["coded"] else (h,)) + _code64(torch.stack([gu[:, :f], gu[:, f:]]), True)
    T, E, k = s["T"], s["E"], s["k"]
    rows = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    n, l = rows.numel(), s["logits"].double()
    top = l.max(1, keepdim=True).values
    ex = torch.exp(l - top)
    lse, p = (top + torch.log(ex.sum(1, keepdim=True)))[:, 0], ex / ex.sum(1, keepdim=True)
    counts = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E)
    f = counts.double() / max(n * k, 1)
    d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    loss = torch.zeros(2, dtype=torch.float64, device="cuda")
    if n:
        loss[0] = s["balance"] * E * (f @ p[rows].mean(0))
        loss[1] = s["z"] * (lse[rows] ** 2).mean()
        pr, up = p[rows], float(s["grad"]) / n
        d[rows] = up * (s["balance"] * E * (pr * f - pr * (pr @ f)[:, None]) + 2 * s["z"] * lse[rows, None] * pr)
    if s["weights"]:
        w, dw = s["w"].double(), s["dw"].double()
        for j in range(k):
            d[torch.arange(T, device="cuda"), s["idx"][:, j].long()] += w[:, j] * (dw[:, j] - (w * dw).sum(1))
    return loss, torch.cat([counts, torch.tensor([n], device="cuda")]).to(torch.int32), d
