"""The 4-bit operators and the token movement over their ranges: rows past 2^31
bytes, dispatch just past the assignments of its one-launch form, the product
at the ends of the scales and on the quantiser's NaN blocks."""

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests import fp4_reference as ref
from tests.test_gpu_fp4_experts import gen, normal, offsets_of, routes

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


# ------------------------------------------------------------------ dispatch

@pytest.mark.parametrize("d,dtype", [(1 << 30, torch.bfloat16), ((1 << 30) + 8, torch.bfloat16), (1 << 29, torch.float32)])
def test_rows_past_32_bits_of_bytes(d, dtype):
    x = torch.zeros(1, d, dtype=dtype, device=DEV)
    x[0, ::4097] = torch.arange(1, -(-d // 4097) + 1, device=DEV).remainder(251).to(dtype)
    idx = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    r = api.dispatch(x, idx, 3)
    assert torch.equal(r.rows[0], x[0]) and torch.equal(r.rows[1], x[0])
    assert r.inv_row.tolist() == [[1, 0]]
    out = api.combine(r.rows, r.inv_row)
    assert torch.equal(out, x + x)


@pytest.mark.parametrize("quantize", [None, "fit"])
@pytest.mark.parametrize("T,k,E,d,dtype", [
    (65, 32, 256, 7168, torch.bfloat16), (70, 31, 40, 1056, torch.float32), (257, 8, 256, 7168, torch.bfloat16),
    (300, 7, 8, 288, torch.bfloat16), (2049, 1, 8, 4096, torch.bfloat16), (1025, 2, 1024, 8224, torch.float32),
    (2500, 3, 5, 32, torch.bfloat16), (700, 3, 16, 16416, torch.bfloat16), (9000, 8, 64, 544, torch.bfloat16)])
def test_tokens_shared_among_ctas(T, k, E, d, dtype, quantize):
    # chunks of few and of many tokens, rows of one piece, of some and of many
    x, idx = normal(T, d, seed=T, dtype=dtype), routes(T, E, k, 0.1, seed=k)
    off, counts, token, inv = ref.maps(idx, E)
    r = api.dispatch(x.to(DEV), idx.to(DEV), E, quantize)
    n = int(off[-1])
    assert torch.equal(r.offsets.cpu(), off) and torch.equal(r.counts.cpu(), counts)
    assert torch.equal(r.row_token.cpu(), token) and torch.equal(r.inv_row.cpu(), inv)
    if quantize is None:
        assert torch.equal(r.rows[:n].cpu(), x[token[:n].long()])
    else:
        codes, scales = (t.cpu() for t in api.quantize_mxfp4(x.to(DEV), quantize))
        assert torch.equal(r.rows[:n].cpu(), codes[token[:n].long()])
        assert torch.equal(r.scales[:n].cpu(), scales[token[:n].long()])


def us_of(*calls, n=20, rounds=9):
    """Median times of the calls on the GPU, each as a graph of n of them, taken in turn."""
    graphs, times, s = [], [[] for _ in calls], torch.cuda.Stream()
    with torch.cuda.stream(s):
        for c in calls:
            c()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for _ in range(n):
                    c()
            g.replay()
            graphs.append(g)
        for _ in range(rounds):
            for g, t in zip(graphs, times):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record(s)
                g.replay()
                b.record(s)
                b.synchronize()
                t.append(1000 * a.elapsed_time(b) / n)
    return [sorted(t)[rounds // 2] for t in times]


@pytest.mark.parametrize("T,k,E,d", [(65, 32, 256, 7168), (257, 8, 256, 7168), (2049, 1, 8, 4096)])
def test_few_long_rows_take_every_sm(T, k, E, d):
    # the same rows by the layer's own permutation, which gives a warp each: a
    # dispatch that leaves SMs idle takes a multiple of its time (65 tokens with
    # 32 rows each on nine CTAs four times), one that takes them all as long
    x, idx = normal(T, d, seed=1).to(DEV), routes(T, E, k, 0.0, seed=2).to(DEV)
    p, R = api.problem(T, d, 128, E, k), T * k
    new = lambda *n, dtype=torch.int32: torch.empty(n, dtype=dtype, device=DEV)  # noqa: E731
    out, rows, work = [new(n) for n in (E, E + 1, R, R)], new(R, d, dtype=x.dtype), api.workspace_for(p)
    mine, other = new(api.moe_dispatch_workspace_size(T, E, k), dtype=torch.uint8), new(R, d, dtype=x.dtype)
    ours, layers = us_of(lambda: api.dispatch(x, idx, E, rows=rows, workspace=mine),
                         lambda: api.moe_permute(p, idx, x, *out, other, work))
    assert torch.equal(rows, other)
    assert ours < 1.5 * layers, (ours, layers)


# ------------------------------------------------------------------- product

KERNELS = pytest.mark.parametrize("count", [4, 100, 300], ids=["few", "some", "many"])
STEP = 2.0 ** -149  # fp32's least


def codes_of(*shape, seed):
    return torch.randint(0, 256, shape, generator=gen(seed), dtype=torch.uint8)


def scales_of(value, *shape):
    return torch.full(shape, value, dtype=torch.uint8)


def multiply(a, sa, w, sw):
    on = [t.to(DEV) for t in (a, sa, offsets_of([a.shape[0]]), w, sw)]
    return api.grouped_mxfp4_gemm(*on, out_dtype=torch.float32).cpu(), ref.product(a, sa, offsets_of([a.shape[0]]), w, sw)[0]


@KERNELS
@pytest.mark.parametrize("sa,sw", [(254, 0), (0, 254), (1, 253), (253, 1), (127, 0), (0, 127), (20, 110), (107, 0), (0, 107), (54, 53)])
def test_product_scale_ends(count, sa, sw):
    # products are multiples of 2^(sa + sw - 256), here at least 2^-149, and a sum
    # of 320 of them is below 2^16 such steps: fp32 holds every partial sum
    K, N = 320, 160
    got, want = multiply(codes_of(count, K // 2, seed=sa), scales_of(sa, count, K // 32), codes_of(1, N, K // 2, seed=sw), scales_of(sw, 1, K // 32, N))
    assert torch.equal(got.double(), want)


@KERNELS
def test_product_every_scale(count):
    # a block's two scales make 1 together: every byte from 0 to 254 in each place
    K, N = 32 * 255, 48
    at = torch.randperm(255, generator=gen(count)).to(torch.uint8)
    got, want = multiply(codes_of(count, K // 2, seed=1), at.expand(count, -1).contiguous(), codes_of(1, N, K // 2, seed=2),
                         (254 - at)[None, :, None].expand(-1, -1, N).contiguous())
    assert torch.equal(got.double(), want)


@KERNELS
def test_product_past_the_largest(count):
    # one code in a row: the result is that code times 2^127, infinite from 2 on
    K, N = 96, 32
    code = torch.zeros(count, K, dtype=torch.uint8)
    code[torch.arange(count), torch.arange(count) % K] = (torch.arange(count) % 16).to(torch.uint8)
    got, want = multiply(ref.pack(code), scales_of(254, count, K // 32), scales_of(0x22, 1, N, K // 2), scales_of(127, 1, K // 32, N))
    assert torch.equal(got, want.float()) and bool(torch.isinf(got).any()) == (count > 4)


@KERNELS
@pytest.mark.parametrize("sa,sw", [(50, 55), (100, 3), (60, 40), (0, 90), (0, 0)])
def test_product_below_the_least_step(count, sa, sw):
    # an instruction loses less than a step of each of its 64 products and of
    # their sum
    K, N = 320, 160
    got, want = multiply(codes_of(count, K // 2, seed=sa), scales_of(sa, count, K // 32), codes_of(1, N, K // 2, seed=sw), scales_of(sw, 1, K // 32, N))
    assert ((got.double() - want).abs() <= 65 * (K // 64) * STEP).all()
    assert sa + sw > 0 or not got.any()


@KERNELS
def test_product_of_values_that_are_not_finite(count):
    # what the quantiser makes of them: the NaN scale and codes of 0, also where
    # the other operand has nothing but zeros
    K, N, E = 320, 160, 2
    x, w = normal(E * count, K, seed=count), normal(E, N, K, seed=count + 1)
    x[:, 96:128], w[:, :, 288:] = 0, 0
    x[1, 40], x[count, 300], w[0, 9, 100], w[1, 77, 5] = float("nan"), float("inf"), float("-inf"), float("nan")
    a, sa = api.quantize_mxfp4(x.to(DEV))
    wq, sw = api.quantize_mxfp4(w.to(DEV), weights=True)
    assert int((sa == 255).sum()) == 2 and not a.cpu()[1, 16:32].any()
    got = api.grouped_mxfp4_gemm(a, sa, offsets_of([count] * E).to(DEV), wq, sw).cpu()
    nan = torch.zeros(E * count, N, dtype=torch.bool)
    nan[1], nan[count], nan[:count, 9], nan[count:, 77] = True, True, True, True
    assert torch.equal(torch.isnan(got), nan) and torch.isfinite(got[~nan]).all()
