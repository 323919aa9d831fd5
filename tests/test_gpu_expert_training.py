"""The expert-training operators against their 64-bit definitions: sizes that
end inside tiles and blocks, experts without rows, rows of no expert, values
that are not finite, and writes outside the outputs."""

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests import train_reference as ref
from tests.guard import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24  # fp32 rounding


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen(seed)).to(dtype)


def offsets_of(counts, first=0):
    o = torch.tensor([first] + list(counts)).cumsum(0)
    return o.to(torch.int32)


def weights(E, N, K, seed=0):
    w = torch.randn(E, N, K, generator=gen(seed)) / K ** 0.5
    codes = torch.empty(E, N, K, dtype=torch.uint8)
    scales = torch.empty(E, ref.blocks(N), ref.blocks(K))
    for i in range(ref.blocks(N)):
        for j in range(ref.blocks(K)):
            b = w[:, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            s = b.abs().amax((1, 2)) / 448
            scales[:, i, j] = s
            codes[:, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = \
                (b / s[:, None, None]).clamp(-448, 448).to(ref.F8).view(torch.uint8)
    return codes, scales


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["amax", "pow2"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 128), (3, 136), (17, 120), (64, 1024), (5, 7168), (2049, 384)])
def test_quantize_blocks_bit_exact(rows, cols, kind, dtype):
    x = normal(rows, cols, seed=rows + cols, dtype=torch.float32) * torch.exp(3 * normal(rows, 1, seed=1, dtype=torch.float32))
    x = x.to(dtype)
    codes, scales = Guarded((rows, cols), torch.uint8, DEV), Guarded((rows, ref.blocks(cols)), torch.float32, DEV)
    api.quantize_blocks(x.to(DEV), kind, codes.t, scales.t)
    c, s = ref.quantize(x, kind)
    assert torch.equal(codes.t.cpu(), c) and torch.equal(scales.t.cpu(), s)
    assert codes.intact() and scales.intact()


@pytest.mark.parametrize("kind", ["amax", "pow2"])
def test_quantize_blocks_special_values(kind):
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(8, 256)
    x[1, 3] = nan
    x[2, :4] = torch.tensor([inf, -inf, 1.5, -3.0])
    x[3] = nan
    x[4, 130] = 448.0
    x[5, 0], x[5, 200] = 3e38, -3e38
    x[6, :3] = torch.tensor([1e-38, -2e-39, 1e-45])  # below the smallest maximum a scale follows
    x[7, ::2] = 1.75
    codes, scales = api.quantize_blocks(x.to(DEV), kind)
    c, s = ref.quantize(x, kind)
    codes, scales = codes.cpu(), scales.cpu()
    assert torch.equal(scales, s) and torch.isfinite(scales).all()
    bad = ~torch.isfinite(x)
    assert ((codes[bad] & 0x7F) == 0x7F).all()
    assert torch.equal(codes[~bad] & 0x7F, c[~bad] & 0x7F)
    assert torch.equal(ref.e4m3(codes)[~bad], ref.e4m3(c)[~bad])


def test_quantize_blocks_takes_rows_that_lie_apart():
    x = normal(33, 640, seed=4).to(DEV)
    got = api.quantize_blocks(x[:, 256:512], "pow2")
    want = api.quantize_blocks(x[:, 256:512].contiguous(), "pow2")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pow2_codes_are_bf16_values():
    x = normal(64, 512, seed=5) * 3
    codes, scales = api.quantize_blocks(x.to(DEV), "pow2")
    v = ref.widen(codes.cpu(), scales.cpu())
    assert torch.equal(v.to(torch.bfloat16).double(), v)


# -------------------------------------------------------------- block product

GEMM = [
    # counts, first row, rows after the last group, K, N
    ([1], 0, 0, 16, 16),
    ([1], 0, 0, 128, 128),
    ([5, 0, 3], 0, 0, 144, 272),
    ([0, 0, 7, 0], 2, 3, 400, 160),
    ([31, 32, 33, 1], 0, 0, 256, 512),
    ([257], 0, 0, 1152, 256),
    ([300, 0, 129, 600], 1, 5, 640, 656),
    ([4500, 70], 0, 0, 128, 304),
    ([2] * 40, 0, 0, 2048, 128),
]


def gemm_case(counts, first, after, K, N, transposed, seed=0):
    E, off = len(counts), offsets_of(counts, first)
    R = int(off[-1]) + after
    a, sa = ref.quantize(normal(R, K, seed=seed), "amax")
    w, sw = weights(E, *((K, N) if transposed else (N, K)), seed=seed + 1)
    return R, a, sa, off, w, sw


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("counts,first,after,K,N", GEMM)
def test_block_gemm(counts, first, after, K, N, transposed, out_dtype):
    R, a, sa, off, w, sw = gemm_case(counts, first, after, K, N, transposed)
    out = Guarded((R, N), out_dtype, DEV)
    out.t.fill_(-77.0)
    api.grouped_block_gemm(a.to(DEV), sa.to(DEV), off.to(DEV), w.to(DEV), sw.to(DEV), transposed, out=out.t)
    got = out.t.cpu().double()
    y, mag = ref.block_gemm(a, sa, off, w, sw, transposed)
    inside = torch.zeros(R, dtype=torch.bool)
    inside[first:first + sum(counts)] = True
    assert (got[~inside] == -77.0).all(), "rows of no expert were written"
    # a block's 128 products in fp32 (at most 16 roundings by twice the unit on
    # the way through the tensor cores), the scales' two and one add a block
    tol = (32 + 4 * ref.blocks(K)) * U * mag + (2.0 ** -8 * y.abs() if out_dtype == torch.bfloat16 else 0)
    assert ((got - y).abs()[inside] <= tol[inside]).all(), float(((got - y).abs() / tol)[inside].max())
    assert out.intact()


@pytest.mark.parametrize("transposed", [False, True], ids=["forward", "gradient"])
def test_block_gemm_keeps_experts_apart(transposed):
    # NaN rows and NaN weights of one expert, and NaN codes next to a matrix's
    # end, reach no other expert's rows; its own rows are NaN
    counts, K, N = [40, 33, 20], 144, 176
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, transposed, seed=3)
    clean = api.grouped_block_gemm(a.to(DEV), sa.to(DEV), off.to(DEV), w.to(DEV), sw.to(DEV), transposed)
    a2, w2 = a.clone(), w.clone()
    a2[40:73] = 0x7F
    w2[1] = 0x7F
    got = api.grouped_block_gemm(a2.to(DEV), sa.to(DEV), off.to(DEV), w2.to(DEV), sw.to(DEV), transposed)
    keep = torch.ones(R, dtype=torch.bool)
    keep[40:73] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert torch.isnan(got[40:73]).all()


def test_block_gemm_many_experts_and_repeat():
    counts = [(7 * e) % 5 if e % 3 else 0 for e in range(1024)]
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, 128, 64, False, seed=5)
    args = [t.to(DEV) for t in (a, sa, off, w, sw)]
    one, two = (api.grouped_block_gemm(*args, out_dtype=torch.float32) for _ in range(2))
    y, mag = ref.block_gemm(a, sa, off, w, sw, False)
    assert ((one.cpu().double() - y).abs() <= 36 * U * mag).all()
    assert torch.equal(one, two)


def test_block_gemm_offsets_out_of_range_are_flagged():
    R, a, sa, off, w, sw = gemm_case([8, 8], 0, 0, 128, 128, False)
    for bad in ([0, 8, 99], [-3, 8, 16], [0, 12, 4]):
        out = Guarded((R, 128), torch.bfloat16, DEV)
        api.grouped_block_gemm(a.to(DEV), sa.to(DEV), torch.tensor(bad, dtype=torch.int32, device=DEV), w.to(DEV),
                               sw.to(DEV), out=out.t)
        assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
        assert out.intact()


def test_block_gemm_data_gradient_is_the_adjoint():
    # <dy, W x> == <W^T dy, x> with the forward's own arrays, in fp32
    counts, K, N = [70, 0, 41], 384, 272
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, False, seed=9)
    d, sd = ref.quantize(normal(R, N, seed=10), "amax")
    dev = [t.to(DEV) for t in (off, w, sw)]
    y = api.grouped_block_gemm(a.to(DEV), sa.to(DEV), *dev, out_dtype=torch.float32).cpu().double()
    dx = api.grouped_block_gemm(d.to(DEV), sd.to(DEV), *dev, transposed=True, out_dtype=torch.float32).cpu().double()
    dy, x = ref.widen(d, sd), ref.widen(a, sa)
    one, two = (dy * y).sum(), (dx * x).sum()
    assert abs(one - two) <= 1e-5 * ((dy * y).abs().sum() + (dx * x).abs().sum())


# --------------------------------------------------------------------- SwiGLU

SWIGLU = [(1, 16), (1, 128), (3, 144), (130, 256), (77, 768), (1031, 384)]


def near_codes(codes, scales, values, dead=0.0):
    """Codes of `values` up to fp32 rounding of the values before the codes':
    within half a step of the code (1/16 of the value, or of the smallest
    step), the scale within 1e-5."""
    top = torch.stack([values[..., b * 128:(b + 1) * 128].abs().amax(-1) for b in range(scales.shape[-1])], -1)
    want = torch.where(top > 0, top.clamp_min(2.0 ** -100) / 448, torch.ones_like(top))
    assert ((scales.double() - want).abs() <= 1e-5 * want).all()
    step = scales.double().repeat_interleave(128, -1)[..., : codes.shape[-1]]
    err = (ref.widen(codes, scales) - values).abs()
    assert (err <= torch.maximum(values.abs() / 16, step * 2.0 ** -10) * (1 + 1e-4) + dead).all()


@pytest.mark.parametrize("apart", [False, True], ids=["dense", "halves"])
@pytest.mark.parametrize("R,f", SWIGLU)
def test_swiglu_save(R, f, apart):
    gu = normal(R, 2 * f, seed=R + f) * 2
    g, u = gu[:, :f], gu[:, f:]
    dev = gu.to(DEV)
    dg, du = (dev[:, :f], dev[:, f:]) if apart else (g.contiguous().to(DEV), u.contiguous().to(DEV))
    r = api.swiglu_save(dg, du, want_h=True)
    h = ref.silu_mul(g.double(), u.double())
    assert ((r.h.cpu().double() - h).abs() <= 2.0 ** -8 * h.abs() + 1e-30).all()
    near_codes(r.codes.cpu(), r.scales.cpu(), h)
    c, s = ref.quantize(torch.stack([g, u]), "pow2")
    assert torch.equal(r.saved.cpu(), c) and torch.equal(r.saved_scales.cpu(), s)


def test_swiglu_outputs_are_optional_and_bounded():
    R, f = 9, 144
    gu = normal(R, 2 * f, seed=8).to(DEV)
    full = api.swiglu_save(gu[:, :f], gu[:, f:], want_h=True)
    only = api.swiglu_save(gu[:, :f], gu[:, f:], want_codes=False)
    assert only.h is None and only.codes is None and torch.equal(only.saved, full.saved)
    out = [Guarded(s, d, DEV) for s, d in (((R, f), torch.bfloat16), ((R, f), torch.uint8), ((R, 2), torch.float32),
                                            ((2, R, f), torch.uint8), ((2, R, 2), torch.float32))]
    api._call("moe_swiglu_save_e4m3", R, f, gu.data_ptr(), gu.data_ptr() + 2 * f, 2 * f,
              *[o.t.data_ptr() for o in out], api._stream(None))
    for o, t in zip(out, full):
        assert torch.equal(o.t, t) and o.intact()


@pytest.mark.parametrize("R,f", SWIGLU)
def test_swiglu_backward(R, f):
    gu = normal(2, R, f, seed=R + f) * 2
    dh = normal(R, f, seed=3)
    saved, scales = ref.quantize(gu, "pow2")
    coded = f % 128 == 0
    r = api.swiglu_backward(saved.to(DEV), scales.to(DEV), dh.to(DEV), want_h=True, want_codes=coded)
    v = ref.widen(saved, scales).requires_grad_()
    h = ref.silu_mul(v[0], v[1])
    h.backward(dh.double())
    want = torch.cat([v.grad[0], v.grad[1]], 1)
    got = r.d_gu.cpu().double()
    # bf16 rounding, and fp32 rounding of 1 + g (1 - sigmoid) where it cancels
    dead = 16 * U * torch.cat([(dh.double() * v[1] * (1 + v[0].abs())).abs(), torch.zeros(R, f, dtype=torch.float64)], 1)
    dead = dead.detach()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + dead).all()
    assert ((r.h.cpu().double() - h.detach()).abs() <= 2.0 ** -8 * h.detach().abs() + 1e-30).all()
    if coded:
        near_codes(r.codes.cpu(), r.scales.cpu(), want, dead)
    else:
        assert r.codes is None


def test_swiglu_backward_against_differences():
    f = 128
    saved, scales = ref.quantize(normal(2, 1, f, seed=2) * 2, "pow2")
    dh = normal(1, f, seed=3)
    r = api.swiglu_backward(saved.to(DEV), scales.to(DEV), dh.to(DEV))
    v, eps = ref.widen(saved, scales), 1e-6
    for part in range(2):
        hi, lo = v.clone(), v.clone()
        hi[part] += eps
        lo[part] -= eps
        diff = (ref.silu_mul(*hi) - ref.silu_mul(*lo)) / (2 * eps) * dh.double()
        got = r.d_gu[:, part * f:(part + 1) * f].cpu().double()
        assert ((got - diff).abs() <= 2.0 ** -8 * diff.abs() + 1e-6).all()


def test_swiglu_extremes():
    # far from zero SiLU is 0 or the identity, and its slope 0 or 1
    g = torch.tensor([[-200.0, -100.0, -90.0, 0.0, -0.0, 90.0, 200.0, 1e30]]).repeat(1, 16).bfloat16()
    u = torch.full_like(g, 2.0)
    r = api.swiglu_save(g.to(DEV), u.to(DEV), want_h=True, want_codes=False)
    want = torch.where(g > 0, 2 * g.float(), torch.zeros_like(g.float()))
    assert torch.equal(r.h.cpu().float(), want)
    g[g == 1e30] = 250.0
    saved, scales = api.quantize_blocks(torch.stack([g, u]).to(DEV), "pow2")
    b = api.swiglu_backward(saved, scales, torch.ones_like(g).to(DEV))
    v = ref.widen(saved.cpu(), scales.cpu())
    sig = 1 / (1 + torch.exp(-v[0]))
    slope = v[1] * sig * (1 + v[0] * (1 - sig))
    # (1e-36 at g = -88: within bf16's rounding, or below fp32's normal range)
    assert ((b.d_gu[:, :128].cpu().double() - slope).abs() <= 2.0 ** -8 * slope.abs() + 2.0 ** -126).all()


# ------------------------------------------------------------ weight gradient

WGRAD = [
    ([1], 0, 0, 16, 16),
    ([3, 0, 17], 0, 0, 144, 272),
    ([0, 64, 0, 65], 5, 9, 256, 128),
    ([15, 16, 129], 0, 3, 400, 656),
    ([700, 256, 257], 1, 0, 272, 304),
    ([4000], 0, 0, 128, 256),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("x_kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("counts,first,after,N,K", WGRAD)
def test_wgrad(counts, first, after, N, K, x_kind, out_dtype):
    E, off = len(counts), offsets_of(counts, first)
    R = int(off[-1]) + after
    dy, x, xs = normal(R, N, seed=1), normal(R, K, seed=2), None
    wide = x.double()
    if x_kind == "e4m3":
        x, xs = ref.quantize(x, "pow2")
        wide = ref.widen(x, xs)
    dw = Guarded((E, N, K), out_dtype, DEV)
    dw.t.fill_(-77.0)
    api.grouped_wgrad(dy.to(DEV), x.to(DEV), None if xs is None else xs.to(DEV), off.to(DEV), dw.t)
    want, mag = ref.wgrad(dy, wide, off)
    got = dw.t.cpu().double()
    # 16 accumulation steps of 16 rows a chunk (each at most twice the unit),
    # and one fp32 add for each chunk of 256 rows
    tol = (40 + max(counts) / 256) * U * mag + (2.0 ** -8 * want.abs() if out_dtype == torch.bfloat16 else 0)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol.clamp_min(1e-30)).max())
    assert dw.intact()


@pytest.mark.parametrize("x_kind", ["e4m3", "bf16"])
def test_wgrad_keeps_experts_apart(x_kind):
    # an expert's rows end inside a stage; what follows there is NaN
    counts, N, K = [37, 50], 144, 160
    off = offsets_of(counts)
    dy, x, xs = normal(87, N, seed=1), normal(87, K, seed=2), None
    if x_kind == "e4m3":
        x, xs = ref.quantize(x, "pow2")
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    clean = api.grouped_wgrad(dev(dy), dev(x), dev(xs), dev(off))
    dy2, x2 = dy.clone(), x.clone()
    dy2[37:], x2[37:] = float("nan"), 0x7F if x_kind == "e4m3" else float("inf")
    got = api.grouped_wgrad(dev(dy2), dev(x2), dev(xs), dev(off))
    assert torch.equal(got[0], clean[0])
    assert torch.isnan(got[1]).all()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_wgrad_accumulates(out_dtype):
    counts, N, K = [20, 0, 300], 144, 272
    off = offsets_of(counts)
    R = sum(counts)
    dy, x = normal(R, N, seed=1).to(DEV), normal(R, K, seed=2).to(DEV)
    start = normal(3, N, K, seed=3, dtype=torch.float32).to(out_dtype)
    fresh = api.grouped_wgrad(dy, x, None, off.to(DEV), dw_dtype=out_dtype).cpu()
    dw = Guarded((3, N, K), out_dtype, DEV, fill=start.to(DEV))
    api.grouped_wgrad(dy, x, None, off.to(DEV), dw.t, accumulate=True)
    assert torch.equal(dw.t.cpu(), (start.float() + fresh.float()).to(out_dtype))
    assert torch.equal(dw.t[1].cpu(), start[1]) and dw.intact()


def test_wgrad_of_half_of_the_rows_columns_and_without_rows():
    off = offsets_of([30, 11]).to(DEV)
    d = normal(41, 512, seed=1).to(DEV)
    x = normal(41, 256, seed=2).to(DEV)
    got = api.grouped_wgrad(d[:, 256:], x, None, off)
    assert torch.equal(got, api.grouped_wgrad(d[:, 256:].contiguous(), x, None, off))
    none = torch.zeros(3, dtype=torch.int32, device=DEV)
    z = api.grouped_wgrad(d[:0], x[:0], None, none, torch.full((2, 512, 256), 5.0, device=DEV))
    assert (z == 0).all()


# --------------------------------------------------------------- router losses

ROUTER = [(1, 2, 1), (5, 8, 2), (64, 8, 2), (33, 60, 4), (17, 128, 8), (300, 130, 6), (1000, 256, 8), (9, 7, 3),
          (41, 33, 32), (50, 1024, 8), (20, 1001, 4), (4097, 16, 2)]


def routed(T, E, k, seed=0):
    logits = 2 * normal(T, E, seed=seed, dtype=torch.float32)
    top, idx = logits.topk(k, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(top, 1)


def close(got, want, rel=1e-5):
    got, want = got.cpu().double(), want.double()
    assert ((got - want).abs() <= rel * want.abs().max() + 1e-30).all(), float((got - want).abs().max())


@pytest.mark.parametrize("masked", [False, True], ids=["all", "masked"])
@pytest.mark.parametrize("T,E,k", ROUTER)
def test_router_losses_and_gradient(T, E, k, masked):
    logits, idx, w = routed(T, E, k, seed=T + E)
    mask = torch.rand(T, generator=gen(1)) < 0.6 if masked else None
    dw = normal(T, k, seed=2, dtype=torch.float32)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    r = api.router_losses(dev(logits), dev(idx), 0.3, 0.02, mask=dev(mask))
    l64 = logits.double().requires_grad_()
    lb, lz, counts = ref.router(l64, idx, mask, 0.3, 0.02)
    close(r.loss[0], lb.detach())
    close(r.loss[1], lz.detach())
    assert torch.equal(r.counts.cpu(), counts)
    close(r.lse, torch.logsumexp(logits.double(), 1))
    grad = torch.tensor([0.7])
    (0.7 * (lb + lz)).backward()
    alone = api.router_losses_backward(dev(logits), dev(idx), r, grad=dev(grad), mask=dev(mask))
    close(alone, l64.grad)
    kept = torch.softmax(l64.gather(1, idx.long()), 1)
    (kept * dw.double()).sum().backward()
    both = api.router_losses_backward(dev(logits), dev(idx), r, grad=dev(grad), topk_w=dev(w), d_topk_w=dev(dw),
                                      mask=dev(mask))
    close(both, l64.grad)
    again = api.router_losses(dev(logits), dev(idx), 0.3, 0.02, mask=dev(mask))
    assert torch.equal(again.loss, r.loss) and torch.equal(again.lse, r.lse)


def test_router_gradient_against_differences():
    T, E, k = 6, 8, 2
    logits, idx, _ = routed(T, E, k, seed=3)
    r = api.router_losses(logits.to(DEV), idx.to(DEV), 1.0, 0.1)
    got = api.router_losses_backward(logits.to(DEV), idx.to(DEV), r).cpu().double()
    for t in range(T):
        for e in range(E):
            v = []
            for d in (1e-5, -1e-5):
                x = logits.double().clone()
                x[t, e] += d
                v.append(sum(ref.router(x, idx, None, 1.0, 0.1)[:2]))
            assert abs((v[0] - v[1]) / 2e-5 - got[t, e]) <= 1e-5 * got.abs().max() + 1e-8


@pytest.mark.parametrize("E", [8, 130])
def test_router_rows_without_probabilities(E):
    # nothing unmasked: no loss, no gradient; a row of -inf adds nothing; an
    # expert masked with -inf or the lowest value gets no probability
    logits, idx, _ = routed(12, E, 2, seed=4)
    none = torch.zeros(12, dtype=torch.bool)
    r = api.router_losses(logits.to(DEV), idx.to(DEV), 1.0, 1.0, mask=none.to(DEV))
    assert (r.loss == 0).all() and (r.counts == 0).all()
    assert (api.router_losses_backward(logits.to(DEV), idx.to(DEV), r, mask=none.to(DEV)) == 0).all()
    low = logits.clone()
    low[:, 1] = -float("inf")
    low[:, 2] = torch.finfo(torch.float32).min
    low[5] = -float("inf")
    r = api.router_losses(low.to(DEV), idx.to(DEV), 1.0, 1.0)
    g = api.router_losses_backward(low.to(DEV), idx.to(DEV), r).cpu()
    assert torch.isfinite(r.loss).all() and torch.isfinite(g).all()
    assert (g[5] == 0).all() and (g[:, 1] == 0).all() and (g[:, 2] == 0).all()
    rest = [t for t in range(12) if t != 5]
    l64 = low[rest].double()
    p, lse = torch.softmax(l64, 1), torch.logsumexp(l64, 1)
    f = torch.bincount(idx.reshape(-1).long(), minlength=E).double() / 24
    close(r.loss[0], E * (f * p.sum(0) / 12).sum())
    close(r.loss[1], (lse * lse).sum() / 12)


def test_router_bad_indices_and_nan():
    logits, idx, w = routed(40, 16, 2, seed=5)
    bad = idx.clone()
    bad[3, 0], bad[7, 1] = 16, -1
    r = api.router_losses(logits.to(DEV), bad.to(DEV), 1.0, 1.0)
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
    assert int(r.counts[:16].sum()) == 78 and int(r.counts[16]) == 40
    api.router_losses_backward(logits.to(DEV), bad.to(DEV), r, topk_w=w.to(DEV), d_topk_w=w.to(DEV))
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
    logits[4, 3] = float("nan")
    r = api.router_losses(logits.to(DEV), idx.to(DEV), 1.0, 1.0)
    g = api.router_losses_backward(logits.to(DEV), idx.to(DEV), r).cpu()
    assert torch.isnan(r.loss).all() and torch.isnan(g[4]).all()
    assert torch.isfinite(g[[t for t in range(40) if t != 4]]).all()


# ------------------------------------------------------------------- streams

def test_operators_run_on_the_stream_they_are_given():
    counts, K, N = [50, 14], 256, 256
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, False, seed=6)
    args = [t.to(DEV) for t in (a, sa, off, w, sw)]
    want = api.grouped_block_gemm(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one = api.grouped_block_gemm(*args)
    two = torch.empty_like(want)
    api.grouped_block_gemm(*args, out=two, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(one, want) and torch.equal(two, want)


def test_operators_in_a_graph():
    counts, K, N = [50, 14], 256, 256
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, False, seed=6)
    a, sa, off, w, sw = (t.to(DEV) for t in (a, sa, off, w, sw))
    x = normal(R, K, seed=7).to(DEV)
    dw = torch.empty(2, N, K, device=DEV)

    def step():
        c, s = api.quantize_blocks(x, "pow2")
        y = api.grouped_block_gemm(c, s, off, w, sw)
        h = api.swiglu_save(y[:, :128], y[:, 128:])
        d = api.swiglu_backward(h.saved, h.saved_scales, y[:, :128].contiguous())
        api.grouped_wgrad(d.d_gu, c, s, off, dw)
        return y, d.d_gu

    step()
    want = [t.clone() for t in (*step(), dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    dw.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, dw), want))


def test_wgrad_multiplies_every_code_out():
    # every E4M3 code under powers of two (small, large, at the edges of what
    # one bf16 product covers) and other scales: dy picks single rows out, so
    # each element is one code times its scale, rounded once to bf16
    K, N = 256, 64
    x = torch.arange(256, dtype=torch.uint8).repeat(N, 1)
    scales = torch.tensor([[2.0 ** (7 - 4 * r), 1.3 * 2.0 ** (r - 40)] for r in range(N)])
    scales[0], scales[1], scales[2] = torch.tensor([2.0 ** 8, 2.0 ** 100]), torch.tensor([2.0 ** -126, 0.0]), -0.5
    dy = torch.eye(N).bfloat16()
    dw = api.grouped_wgrad(dy.to(DEV), x.to(DEV), scales.to(DEV), offsets_of([N]).to(DEV)).cpu()[0]
    s = scales.repeat_interleave(128, 1)
    want = (ref.e4m3(x).float() * s).bfloat16().float()
    # (a NaN code reaches every n of its column: 0 * NaN is NaN)
    nan = torch.isnan(want).any(0)
    assert torch.equal(nan, torch.tensor([c % 128 == 127 for c in range(256)]))
    assert torch.isnan(dw[:, nan]).all()
    assert torch.equal(dw[:, ~nan], want[:, ~nan])


@pytest.mark.parametrize("transposed", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("K", [128, 384, 656])
def test_block_gemm_tiles_of_every_size_in_turn(K, transposed):
    # tiles with many rows and with few alternate on every CTA, so that the
    # accumulators change hands again and again; blocks in no multiple of four
    counts = [[300, 5, 97, 40, 96, 256, 1, 130, 70, 33, 0, 512, 64][i % 13] for i in range(130)]
    N = 512
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, transposed, seed=K)
    args = [t.to(DEV) for t in (a, sa, off, w, sw)]
    got = api.grouped_block_gemm(*args, transposed, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(api.grouped_block_gemm(*args, transposed, out_dtype=torch.float32), got)
    y, mag = ref.block_gemm(a, sa, off, w, sw, transposed)
    assert ((got.cpu().double() - y).abs() <= (32 + 4 * ref.blocks(K)) * U * mag).all()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("K,N", [(16, 16), (144, 1296), (640, 400), (1152, 272)])
def test_block_gemm_many_rows_an_expert(K, N, transposed, out_dtype):
    # several tiles an expert on average, groups and matrices that end
    # anywhere in one, and more units than CTA pairs
    counts = [700, 0, 257, 1, 900, 385, 31, 5200, 33]
    R, a, sa, off, w, sw = gemm_case(counts, 3, 2, K, N, transposed, seed=K)
    assert R >= 256 * len(counts)
    args = [t.to(DEV) for t in (a, sa, off, w, sw)]
    out = Guarded((R, N), out_dtype, DEV)
    out.t.fill_(-77.0)
    api.grouped_block_gemm(*args, transposed, out=out.t)
    got = out.t.clone()
    for _ in range(10):
        api.grouped_block_gemm(*args, transposed, out=out.t)
        assert torch.equal(out.t, got)
    got = got.cpu().double()
    y, mag = ref.block_gemm(a, sa, off, w, sw, transposed)
    inside = torch.zeros(R, dtype=torch.bool)
    inside[3:3 + sum(counts)] = True
    assert (got[~inside] == -77.0).all(), "rows of no expert were written"
    tol = (32 + 4 * ref.blocks(K)) * U * mag + (2.0 ** -8 * y.abs() if out_dtype == torch.bfloat16 else 0)
    assert ((got - y).abs()[inside] <= tol[inside]).all(), float(((got - y).abs() / tol)[inside].max())
    assert out.intact()


@pytest.mark.parametrize("transposed", [False, True], ids=["forward", "gradient"])
def test_block_gemm_many_rows_keep_experts_apart(transposed):
    counts, K, N = [400, 333, 290], 144, 176
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, transposed, seed=3)
    clean = api.grouped_block_gemm(a.to(DEV), sa.to(DEV), off.to(DEV), w.to(DEV), sw.to(DEV), transposed)
    a2, sa2, w2 = a.clone(), sa.clone(), w.clone()
    a2[400:733] = 0x7F
    sa2[400:733] = float("inf")
    w2[1] = 0x7F
    got = api.grouped_block_gemm(a2.to(DEV), sa2.to(DEV), off.to(DEV), w2.to(DEV), sw.to(DEV), transposed)
    keep = torch.ones(R, dtype=torch.bool)
    keep[400:733] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert torch.isnan(got[400:733]).all()
