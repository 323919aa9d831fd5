"""The 4-bit operators and the token movement against their definitions: sizes
that end inside blocks, tiles and chunks, experts without rows, dropped
assignments, values that are not finite, and writes outside the outputs."""

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests import fp4_reference as ref
from tests.guard import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24  # fp32 rounding
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}  # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(*shape, seed=0, dtype=torch.bfloat16):
    g = gen(seed)
    x = torch.randn(*shape, generator=g)
    return (x * torch.exp(torch.randn(*shape[:-1], 1, generator=g))).to(dtype)


def offsets_of(counts, first=0):
    return torch.tensor([first] + list(counts)).cumsum(0).to(torch.int32)


def same(a, b):
    """Equal bits, but any NaN for any other."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ----------------------------------------------------------- quantise, values

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["floor", "fit"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 1056), (64, 2048), (1049, 64), (5, 7168)])
def test_quantize_rows_bit_exact(rows, cols, kind, dtype):
    x = normal(rows, cols, seed=rows + cols, dtype=TYPES[dtype])
    codes, scales = Guarded((rows, cols // 2), torch.uint8, DEV), Guarded((rows, cols // 32), torch.uint8, DEV)
    api.quantize_mxfp4(x.to(DEV), kind, codes=codes.t, scales=scales.t)
    c, s = ref.quantize(x, kind)
    assert torch.equal(scales.t.cpu(), s) and torch.equal(codes.t.cpu(), c)
    assert codes.intact() and scales.intact()
    for t in TYPES.values():
        out = Guarded((rows, cols), t, DEV)
        api.mxfp4_values(codes.t, scales.t, out=out.t)
        assert torch.equal(out.t.cpu().double(), ref.widen(c, s)) and out.intact()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,N,K", [(1, 16, 32), (3, 48, 1056), (2, 80, 2080), (1, 304, 64), (1, 1, 32), (3, 17, 96), (2, 33, 1088),
                                   (5, 30, 64), (2, 100, 32)])
def test_quantize_weights_bit_exact(E, N, K, dtype):
    x = normal(E, N, K, seed=N + K, dtype=TYPES[dtype])
    codes, scales = Guarded((E, N, K // 2), torch.uint8, DEV), Guarded((E, K // 32, N), torch.uint8, DEV)
    api.quantize_mxfp4(x.to(DEV), weights=True, codes=codes.t, scales=scales.t)
    c, s = ref.quantize(x, "floor")
    assert torch.equal(codes.t.cpu(), c) and torch.equal(scales.t.cpu(), s.transpose(1, 2))
    assert codes.intact() and scales.intact()
    out = Guarded((E, N, K), TYPES[dtype], DEV)
    api.mxfp4_values(codes.t, scales.t, weights=True, out=out.t)
    assert torch.equal(out.t.cpu().double(), ref.widen(c, s)) and out.intact()


@pytest.mark.parametrize("kind", ["floor", "fit"])
def test_quantize_every_rounding_and_special_values(kind):
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(16, 32)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])  # every tie, and next to it on either side
    x[0] = torch.cat([mid, -mid, torch.nextafter(mid, torch.tensor(9.0)), torch.nextafter(mid, torch.tensor(0.0)),
                      torch.tensor([6.0, -0.0, 0.0, 4.0])])
    x[1], x[2] = x[0] * 2.0 ** 60, x[0] * 2.0 ** -60
    x[3, :4] = torch.tensor([7.999, 6.0, 6.001, -7.0])   # above 6 scales (floor), above 3 (fit)
    x[4, 0], x[5, 0], x[5, 1], x[6] = nan, inf, 3.0, -inf
    x[7, 0], x[7, 1] = 3.4e38, -1e38
    x[8, :3] = torch.tensor([1e-38, -2e-39, 1e-45])     # the least scale
    x[9, 5] = 1e-45
    x[10] = -0.0
    x[11, :2] = torch.tensor([2.0 ** -125, 2.0 ** -126])
    x[12, 0] = 2.0 ** -124
    x[13] = 6.0 * 2.0 ** torch.arange(-16, 16).float()
    c, s = ref.quantize(x, kind)
    codes, scales = (t.cpu() for t in api.quantize_mxfp4(x.to(DEV), kind))
    assert torch.equal(scales, s) and torch.equal(codes, c)
    assert [int(v) for v in s[4:7, 0]] == [255] * 3 and int(s[10, 0]) == 127
    # bf16 has the same exponents
    b = x.bfloat16()
    c, s = ref.quantize(b, kind)
    codes, scales = (t.cpu() for t in api.quantize_mxfp4(b.to(DEV), kind))
    assert torch.equal(scales, s) and torch.equal(codes, c)


def test_values_of_every_code_and_scale():
    codes = ref.pack(torch.arange(16, dtype=torch.uint8).repeat(256, 2))
    scales = torch.arange(256).to(torch.uint8)[:, None].contiguous()
    want = ref.widen(codes, scales)
    for t in TYPES.values():
        got = api.mxfp4_values(codes.to(DEV), scales.to(DEV), dtype=t).cpu()
        assert same(got, want.to(torch.float32).to(t))


@pytest.mark.parametrize("shift", [0, 8, 16, 40])
def test_quantize_takes_rows_that_lie_apart_and_other_shapes(shift):
    x = normal(33, 640, seed=4).to(DEV)
    part = x[:, shift:shift + 256]
    got, want = api.quantize_mxfp4(part), api.quantize_mxfp4(part.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    three = x[:32].view(4, 8, 640)
    got, want = api.quantize_mxfp4(three), api.quantize_mxfp4(x[:32])
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    turned = three.transpose(0, 1)
    got, want = api.quantize_mxfp4(turned), api.quantize_mxfp4(turned.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# --------------------------------------------------------------------- SwiGLU

@pytest.mark.parametrize("kind", ["floor", "fit"])
@pytest.mark.parametrize("R,f", [(1, 32), (7, 96), (33, 768), (1048, 160)])
def test_swiglu(R, f, kind):
    gu = normal(R, 2 * f, seed=R)
    g, u = gu[:, :f].double(), gu[:, f:].double()
    h = g / (1 + torch.exp(-g)) * u
    got = api.swiglu_mxfp4(gu.to(DEV)[:, :f], gu.to(DEV)[:, f:], kind, want_h=True)
    # h in fp32: the sigmoid is within 2^-18 (its exponential's 28 units of
    # 2^-23 at the worst, the reciprocal's 1 and three roundings, with room)
    off = 2.0 ** -18
    assert ((got.h.cpu().double() - h).abs() <= (off + 2.0 ** -8) * h.abs() + 1e-37).all()
    # codes: those of some value that near, by the block's own scale; the scale
    # that of some maximum that near
    lo, hi = h.abs() * (1 - off), h.abs() * (1 + off)
    s_lo, s_hi = ref.quantize(lo, kind)[1], ref.quantize(hi, kind)[1]
    s = got.scales.cpu()
    assert ((s == s_lo) | (s == s_hi)).all()
    v = ref.widen(got.codes.cpu(), s)
    scale = torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    code = lambda y: ref.E2M1[:8][((y / scale)[..., None] > torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],  # noqa: E731
                                                                        dtype=torch.float64)).sum(-1)]
    assert ((v.abs() >= code(lo) * scale - 1e-300) & (v.abs() <= code(hi * (1 + 1e-12)) * scale)).all()
    assert (torch.sign(v) * torch.sign(h) >= 0).all()


def test_swiglu_special_values():
    gu = torch.zeros(4, 64, dtype=torch.bfloat16)
    gu[0, 0], gu[0, 32] = float("nan"), 1.0
    gu[1, 0], gu[1, 32] = float("inf"), 1.0
    gu[2, 0], gu[2, 32], gu[2, 1], gu[2, 33] = -300.0, 1.0, 2.0, 2.0  # a gate so low that nothing is left
    got = api.swiglu_mxfp4(gu.to(DEV)[:, :32], gu.to(DEV)[:, 32:])
    s = got.scales.cpu().flatten().tolist()
    assert s[:2] == [255, 255] and s[3] == 127
    v = ref.widen(got.codes.cpu(), got.scales.cpu())
    assert v[2, 0] == 0 and abs(float(v[2, 1]) - 4 / (1 + 2.718281828 ** -2.0)) <= 0.6 and (v[3] == 0).all()


# ------------------------------------------------------------------- dispatch

def routes(T, E, k, drop, seed=0):
    g = gen(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32) if E >= k else \
        torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    return torch.where(torch.rand(T, k, generator=g) < drop, torch.full_like(idx, -1), idx).contiguous()


DISPATCH = [
    # T, E, k, d, dropped
    (1, 1, 1, 8, 0.0),
    (1, 256, 8, 64, 0.0),
    (5, 8, 2, 1056, 0.3),
    (64, 256, 8, 96, 0.0),
    (130, 1024, 3, 32, 0.1),
    (7, 4, 4, 2048, 1.0),      # nothing is left
    (64, 1024, 32, 32, 0.1),   # the most slots; 2048 assignments, the last of the one launch
    (683, 16, 3, 32, 0.0),     # 2049
    (700, 1000, 7, 96, 0.2),
    (3000, 2, 1, 64, 0.5),
    (2100, 128, 8, 32, 0.07),
    (90, 3, 30, 32, 0.1),      # an expert more than once in a token
    (4000, 33, 5, 8, 0.9),
    (70000, 40, 2, 8, 0.05),   # slices of more chunks than registers hold
    (1905, 610, 1, 32, 0.0),   # shared memory just below the 48 KB that need no asking
    (2041, 602, 1, 32, 0.0),
]


@pytest.mark.parametrize("T,E,k,d,drop", DISPATCH)
@pytest.mark.parametrize("to", ["bf16", "f32", "bf16-floor", "f32-fit"])
def test_dispatch(T, E, k, d, drop, to):
    t, mx = TYPES[to.split("-")[0]], to.split("-")[1] if "-" in to else None
    if mx and d % 32:
        pytest.skip("MXFP4 rows have blocks of 32")
    x, idx, R = normal(T, d, seed=T, dtype=t), routes(T, E, k, drop, seed=T + E), T * k
    n = 2 if mx else 1
    rows = Guarded((R, d // n), torch.uint8 if mx else t, DEV, fill=7)
    scales = Guarded((R, d // 32), torch.uint8, DEV, fill=9) if mx else None
    got = api.dispatch(x.to(DEV), idx.to(DEV), E, quantize=mx, rows=rows.t, scales=scales.t if mx else None)
    offsets, counts, token, inv = ref.maps(idx, E)
    for a, b in zip((got.offsets, got.counts, got.row_token, got.inv_row), (offsets, counts, token, inv)):
        assert torch.equal(a.cpu(), b)
    live = int(offsets[-1])
    source = x[token[:live].long()]
    if mx:
        c, s = ref.quantize(x, mx)
        assert torch.equal(scales.t[:live].cpu(), s[token[:live].long()]) and bool((scales.t[live:] == 9).all()) and scales.intact()
        source = c[token[:live].long()]
    assert torch.equal(rows.t[:live].cpu(), source) and bool((rows.t[live:] == 7).all()) and rows.intact()
    # the maps alone
    alone = api.dispatch(None, idx.to(DEV), E)
    assert alone.rows is None and all(torch.equal(a, b) for a, b in zip(alone[2:], got[2:]))


def test_dispatch_rows_that_lie_apart():
    x, idx = normal(300, 256, seed=1).to(DEV), routes(300, 8, 2, 0.1).to(DEV)
    for shift in (0, 8, 24):
        part = x[:, shift:shift + 96]
        for mx in (None, "floor"):
            n = int(ref.maps(idx.cpu(), 8)[0][-1])
            a, b = api.dispatch(part, idx, 8, mx), api.dispatch(part.contiguous(), idx, 8, mx)
            assert torch.equal(a.rows[:n], b.rows[:n]) and (mx is None or torch.equal(a.scales[:n], b.scales[:n]))


def test_dispatch_without_tokens():
    got = api.dispatch(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV), 5)
    assert got.offsets.tolist() == [0] * 6 and got.counts.tolist() == [0] * 5 and got.rows.shape == (0, 64)


@pytest.mark.parametrize("T", [40, 4000])
def test_dispatch_flags_experts_out_of_range(T):
    x, idx = normal(T, 32, seed=2), routes(T, 8, 2, 0.1)
    bad = idx.clone()
    bad[3, 1], bad[T - 1, 0] = 8, 2 ** 31 - 1
    got = api.dispatch(x.to(DEV), bad.to(DEV), 8)
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
    idx[3, 1] = idx[T - 1, 0] = -1
    want = ref.maps(idx, 8)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got[2:], want))


# -------------------------------------------------------------------- combine

COMBINE = [
    # T, k, d, R more than assigned, dropped
    (1, 1, 8, 0, 0.0),
    (1, 8, 7168, 0, 0.0),
    (6, 3, 264, 4, 0.3),
    (65, 8, 512, 0, 0.1),
    (300, 2, 1032, 9, 0.5),
    (33, 9, 96, 0, 0.1),
    (20, 32, 64, 0, 0.2),
    (4, 4, 2048, 0, 1.0),
    (2600, 1, 264, 0, 0.1),
    (2500, 2, 1032, 3, 0.2),
    (2450, 4, 520, 0, 0.0),
    (2440, 7, 136, 1, 0.1),
    (2433, 11, 72, 0, 0.3),
]


def inverse(T, k, more, drop, seed):
    """Rows at random places, with some that no assignment has."""
    R = T * k + more
    inv = torch.randperm(R, generator=gen(seed))[: T * k].view(T, k).to(torch.int32)
    return torch.where(torch.rand(T, k, generator=gen(seed + 1)) < drop, torch.full_like(inv, -1), inv), R


@pytest.mark.parametrize("T,k,d,more,drop", COMBINE)
@pytest.mark.parametrize("dtype", TYPES)
def test_combine(T, k, d, more, drop, dtype):
    t = TYPES[dtype]
    inv, R = inverse(T, k, more, drop, seed=T + d)
    y, add, w = normal(R, d, seed=1, dtype=t), normal(T, d, seed=2, dtype=t), torch.rand(T, k, generator=gen(3))
    for wi, ai in ((w, add), (w, None), (None, add), (None, None)):
        want, mag = ref.combine(y, inv, wi, ai)
        out = Guarded((T, d), t, DEV)
        args = [v if v is None else v.to(DEV) for v in (y, inv, wi, ai)]
        api.combine(*args, out=out.t)
        # k fused products and a sum in fp32 in turn, then the output's rounding
        tol = (k + 1) * U * mag * (1 + 2.0 ** -7) + HALF[t] * want.abs()
        assert ((out.t.cpu().double() - want).abs() <= tol).all() and out.intact()
        if wi is None:
            assert torch.equal(api.dispatch_backward(args[0], args[1], args[3]), out.t)
    dest = add.to(DEV)
    on = [v.to(DEV) for v in (y, inv, w)]
    want = api.combine(*on, add.to(DEV))
    assert torch.equal(api.combine(*on, dest, out=dest), want)


@pytest.mark.parametrize("T,k,d,more,drop", COMBINE)
@pytest.mark.parametrize("dtype", TYPES)
def test_combine_backward(T, k, d, more, drop, dtype):
    t = TYPES[dtype]
    inv, R = inverse(T, k, more, drop, seed=T + d)
    y, d_out, w = normal(R, d, seed=1, dtype=t), normal(T, d, seed=2, dtype=t), torch.rand(T, k, generator=gen(3))
    on = [v.to(DEV) for v in (d_out, y, inv, w)]
    for wi in (w, None):
        dy, dw, mag = ref.combine_backward(d_out, y, inv, wi)
        out = Guarded((R, d), t, DEV, fill=5)
        got = api.combine_backward(*on[:3], None if wi is None else on[3], dy=out.t)
        mine = ~torch.isnan(dy).all(1)
        assert bool((out.t.cpu()[~mine] == 5).all()) and out.intact()
        # one product in fp32 and the output's rounding
        assert ((out.t.cpu().double()[mine] - dy[mine]).abs() <= (U + HALF[t]) * (1 + U) * dy[mine].abs()).all()
        # d fused products and sums in fp32: a lane's own in turn, which are d / 32
        # (up to 8 more where d ends inside a warp's piece) where a warp takes a
        # token and fewer where a CTA does, then five sums over lanes and four
        # over warps
        assert ((got.dw.cpu().double() - dw).abs() <= (d // 32 + 20) * U * mag).all()
        one = api.combine_backward(*on[:3], None if wi is None else on[3], want_dw=False)
        assert one.dw is None and torch.equal(one.dy[mine.to(DEV)], out.t[mine.to(DEV)])
        other = api.combine_backward(*on, want_dy=False)
        assert other.dy is None and torch.equal(other.dw, got.dw)


def test_combine_gradients_against_differences():
    # combine is linear in the rows and in the weights: a difference over any
    # step is the derivative, but for fp32's rounding
    T, k, d = 9, 3, 128
    inv, R = inverse(T, k, 2, 0.2, 5)
    y, w, c = normal(R, d, seed=1, dtype=torch.float32), torch.rand(T, k, generator=gen(2)), normal(T, d, seed=3, dtype=torch.float32)
    loss = lambda y, w: float((ref.combine(y, inv, w)[0] * c.double()).sum())  # noqa: E731
    got = api.combine_backward(c.to(DEV), y.to(DEV), inv.to(DEV), w.to(DEV), dy=torch.zeros(R, d, device=DEV))
    dy, dw = got.dy.cpu(), got.dw.cpu()
    for _ in range(20):
        r, i, t, j = (int(torch.randint(n, (1,), generator=gen(_ * 7 + q))) for q, n in enumerate((R, d, T, k)))
        up, uw = y.clone(), w.clone()
        up[r, i] += 1
        uw[t, j] += 1
        scale = float((c.abs().sum() * (1 + y.abs().max())))
        assert abs(loss(up, w) - loss(y, w) - float(dy[r, i])) <= 1e-6 * scale
        assert abs(loss(y, uw) - loss(y, w) - float(dw[t, j])) <= 1e-6 * scale


def test_combine_flags_rows_out_of_range():
    y, inv = normal(6, 64, seed=1), torch.tensor([[0, 6], [5, -1]], dtype=torch.int32)
    out = api.combine(y.to(DEV), inv.to(DEV))
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
    assert torch.equal(out.cpu(), y[[0, 5]])
    api.combine_backward(y[:2].to(DEV), y.to(DEV), inv.to(DEV))
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS


def test_dispatch_and_combine_are_each_others_gradient():
    # <combine(dispatch(x)), c> with weights, against autograd on the plain form
    T, E, k, d = 50, 8, 3, 64
    idx = routes(T, E, k, 0.2, seed=4)
    x, w, c = (normal(*s, seed=i, dtype=torch.float32) for i, s in enumerate(((T, d), (T, k), (T, d))))
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    on = (idx >= 0).double()
    (xd * (wd * on).sum(1, keepdim=True) * c.double()).sum().backward()
    r = api.dispatch(x.to(DEV), idx.to(DEV), E)
    g = api.combine_backward(c.to(DEV), r.rows, r.inv_row, w.to(DEV))
    dx = api.dispatch_backward(g.dy, r.inv_row).cpu().double()
    mag = (w.abs() * on).sum(1, keepdim=True).double() * c.abs().double()
    assert ((dx - xd.grad).abs() <= (k + 2) * U * mag).all()
    dw_mag = (x.abs().double() * c.abs().double()).sum(1, keepdim=True)
    assert ((g.dw.cpu().double() - wd.grad).abs() <= 28 * U * dw_mag).all()


# -------------------------------------------------------------------- product

def product_case(counts, first, after, K, N, seed=0, kind="floor"):
    E, off = len(counts), offsets_of(counts, first)
    R = int(off[-1]) + after
    a, sa = ref.quantize(normal(R, K, seed=seed), kind)
    w, sw = ref.quantize(normal(E, N, K, seed=seed + 1), kind)
    return R, a, sa, off, w, sw.transpose(1, 2).contiguous()


def near(got, y, mag, K, dtype):
    # an instruction adds 64 exact products to the sum and keeps at least
    # fp32's bits of the largest term: 4 units of 2^-24 of the terms'
    # magnitude for each, and the output's rounding
    tol = (32 + 4 * -(-K // 64)) * U * mag + (HALF[dtype] * y.abs() if dtype == torch.bfloat16 else 0)
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float(((got.double() - y).abs() / tol).max()))


PRODUCT = [
    # counts, first row, rows after the last group, K, N
    ([1], 0, 0, 32, 16),
    ([1], 0, 0, 256, 128),
    ([8], 0, 0, 64, 128),
    ([5, 0, 3], 0, 0, 160, 272),
    ([0, 0, 7, 0], 2, 3, 416, 160),
    ([31, 32, 33, 1], 0, 0, 256, 512),
    ([65, 64, 63], 0, 0, 512, 144),
    ([257], 0, 0, 1152, 256),
    ([300, 0, 129, 600], 1, 5, 672, 656),
    ([4500, 70], 0, 0, 128, 304),
    ([2] * 40, 0, 0, 2048, 128),
    ([130, 250, 512], 0, 0, 768, 384),
    # many rows: ends inside a tile, next to one, at one, short and long reductions
    ([300, 0, 113, 256, 511], 3, 2, 256, 240),
    ([256, 129], 0, 0, 96, 480),
    ([700], 0, 1, 544, 496),
    ([400, 150], 0, 0, 1280, 256),
    ([260, 300], 0, 0, 2592, 496),
    ([1100], 0, 0, 1024, 16),
]


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("counts,first,after,K,N", PRODUCT)
def test_product(counts, first, after, K, N, out_dtype):
    t = TYPES[out_dtype]
    R, a, sa, off, w, sw = product_case(counts, first, after, K, N, seed=K + N)
    y, mag = ref.product(a, sa, off, w, sw)
    out = Guarded((R, N), t, DEV, fill=3)
    api.grouped_mxfp4_gemm(*(v.to(DEV) for v in (a, sa, off, w, sw)), out=out.t)
    got = out.t.cpu()
    inside = ~torch.isnan(y).all(1)
    assert bool((got[~inside] == 3).all()) and out.intact()
    near(got[inside], y[inside], mag[inside], K, t)


def test_product_single_codes():
    # one code at a time: every place of a row and of the weights' reduction
    # meets its own code and scale
    K, N, R = 512, 128, 64
    g = gen(7)
    a = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    sa = torch.randint(100, 140, (R, K // 32), generator=g, dtype=torch.uint8)
    code = torch.zeros(1, N, K, dtype=torch.uint8)
    at = torch.randperm(K, generator=g)[:N]
    code[0, torch.arange(N), at] = 2  # 1.0
    w, sw = ref.pack(code), torch.randint(110, 140, (1, K // 32, N), generator=g, dtype=torch.uint8)
    off = offsets_of([R])
    got = api.grouped_mxfp4_gemm(*(v.to(DEV) for v in (a, sa, off, w, sw)), out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), ref.product(a, sa, off, w, sw)[0])


@pytest.mark.parametrize("count", [3, 40, 120, 300])
def test_product_into_rows_that_lie_apart(count):
    R, a, sa, off, w, sw = product_case([count], 0, 0, 256, 144, seed=count)
    on = [v.to(DEV) for v in (a, sa, off, w, sw)]
    want = api.grouped_mxfp4_gemm(*on)
    both = torch.full((R, 400), 3.0, dtype=torch.bfloat16, device=DEV)
    api.grouped_mxfp4_gemm(*on, out=both[:, 200:344])
    assert torch.equal(both[:, 200:344], want) and bool((both[:, :200] == 3).all()) and bool((both[:, 344:] == 3).all())


@pytest.mark.parametrize("count", [5, 100, 300])
def test_product_keeps_nan_to_its_rows_and_channels(count):
    R, a, sa, off, w, sw = product_case([count, count], 0, 0, 320, 160, seed=count)
    sa[2, 3], sw[1, 9, 40] = 255, 255
    y, mag = ref.product(a, sa, off, w, sw)
    got = api.grouped_mxfp4_gemm(*(v.to(DEV) for v in (a, sa, off, w, sw))).cpu()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan) and nan[2].all() and nan[count:, 40].all() and int(nan.sum()) == 160 + count
    near(got[~nan], y[~nan], mag[~nan], 320, torch.bfloat16)


@pytest.mark.parametrize("R,bad,good", [(12, [-3, 4, 2, 40], [0, 4, 4, 12]), (500, [-9, 300, 200, 5000], [0, 300, 300, 500]),
                                        (150, [0, 90, 2 ** 31 - 1, -2 ** 31], [0, 90, 150, 150])])
def test_product_clamps_offsets_out_of_range(R, bad, good):
    _, a, sa, _, w, sw = product_case([R, 0, 0], 0, 0, 64, 32)
    got = api.grouped_mxfp4_gemm(*(v.to(DEV) for v in (a, sa, torch.tensor(bad, dtype=torch.int32), w, sw)), out_dtype=torch.float32)
    assert api.moe_read_device_status() == api.ERR_DEVICE_BOUNDS
    y, mag = ref.product(a, sa, torch.tensor(good, dtype=torch.int32), w, sw)
    near(got.cpu(), y, mag, 64, torch.float32)


@pytest.mark.parametrize("E,rows,empty", [(1024, 3, 0.7), (1000, 120, 0.6), (1024, 600, 0.5), (333, 400, 0.1)])
def test_product_many_experts(E, rows, empty):
    # (few, some and many rows an expert on average; long stretches without any)
    g = gen(E + rows)
    counts = torch.randint(1, 2 * rows, (E,), generator=g)
    counts[torch.rand(E, generator=g) < empty] = 0
    counts[E // 3:E // 3 + 70] = 0
    off = offsets_of(counts.tolist())
    R, K, N = int(off[-1]), 64, 48
    a, sa = api.quantize_mxfp4(normal(R, K, seed=1).to(DEV))
    w, sw = api.quantize_mxfp4(normal(E, N, K, seed=2).to(DEV), weights=True)
    got = api.grouped_mxfp4_gemm(a, sa, off.to(DEV), w, sw).cpu()
    y, mag = ref.product(a.cpu(), sa.cpu(), off, w.cpu(), sw.cpu())
    near(got, y, mag, K, torch.bfloat16)


def test_product_without_rows():
    _, a, sa, off, w, sw = product_case([1], 0, 0, 64, 32)
    on = [v.to(DEV) for v in (a, sa, off, w, sw)]
    assert api.grouped_mxfp4_gemm(on[0][:0], on[1][:0], *on[2:]).shape == (0, 32)
    out = torch.full((1, 32), 3.0, dtype=torch.bfloat16, device=DEV)
    api.grouped_mxfp4_gemm(on[0], on[1], torch.zeros(2, dtype=torch.int32, device=DEV), *on[3:], out=out)
    assert bool((out == 3).all())
