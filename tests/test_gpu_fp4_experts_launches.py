"""The 4-bit operators and the token movement launched in other ways than one
call at a time on the current stream: together as a layer uses them, in quick
succession, in captured graphs, on given streams, from several threads, on
results past 2^31 elements, under a short limit of waits."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build
from tests import fp4_reference as ref
from tests.test_gpu_expert_training_launches import ENDS, check_on_stream, ends_of, tall
from tests.test_gpu_fp4_experts import U, gen, near, normal, offsets_of, product_case, routes

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


def weights(E, N, K, seed):
    w, s = ref.quantize(torch.randn(E, N, K, generator=gen(seed)).bfloat16() / K ** 0.5, "floor")
    return w, s.transpose(1, 2).contiguous()


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("T,d,ffn,E,k,drop", [(1, 256, 128, 8, 2, 0.0), (37, 256, 96, 4, 2, 0.2), (700, 160, 64, 16, 3, 0.1),
                                             (900, 128, 128, 2, 1, 0.0)])
def test_layer_in_4_bits(T, d, ffn, E, k, drop):
    # each stage against the definition on what the stage before returned
    x, idx, w = normal(T, d, seed=1), routes(T, E, k, drop, seed=2), torch.rand(T, k, generator=gen(3))
    shared = normal(T, d, seed=4)
    (wg, sg), (wd, sd) = weights(E, 2 * ffn, d, 5), weights(E, d, ffn, 6)
    on = [t.to(DEV) for t in (x, idx, w, shared, wg, sg, wd, sd)]
    r = api.dispatch(on[0], on[1], E, quantize="floor")
    gu = api.grouped_mxfp4_gemm(r.rows, r.scales, r.offsets, on[4], on[5])
    h = api.swiglu_mxfp4(gu[:, :ffn], gu[:, ffn:], "fit")
    y = api.grouped_mxfp4_gemm(h.codes, h.scales, r.offsets, on[6], on[7], out_dtype=torch.float32)
    out = api.combine(y.bfloat16(), r.inv_row, on[2], add=on[3])
    off, counts, token, inv = ref.maps(idx, E)
    n = int(off[-1])
    assert torch.equal(r.offsets.cpu(), off) and torch.equal(r.inv_row.cpu(), inv)
    c, s = ref.quantize(x, "floor")
    want, mag = ref.product(c[token[:n].long()], s[token[:n].long()], off, wg, sg)
    near(gu[:n].cpu(), want, mag, d, torch.bfloat16)
    want, mag = ref.product(h.codes[:n].cpu(), h.scales[:n].cpu(), off, wd, sd)
    near(y[:n].cpu(), want, mag, ffn, torch.float32)
    rows = torch.zeros(T * k, d, dtype=torch.bfloat16)
    rows[:n] = y[:n].cpu().bfloat16()
    want, mag = ref.combine(rows, inv, w, shared)
    assert ((out.cpu().double() - want).abs() <= (k + 2) * U * mag + 2.0 ** -8 * want.abs()).all()


def test_gradient_of_the_rows_by_the_same_product():
    # dx = dy W: the product with the codes of each matrix's transpose
    E, N, K, counts = 3, 96, 160, [40, 0, 33]
    w = torch.randn(E, N, K, generator=gen(1)).to(DEV)
    wt, st = api.quantize_mxfp4(w.transpose(1, 2), weights=True)
    dy = normal(73, N, seed=2).to(DEV)
    a, sa = api.quantize_mxfp4(dy)
    off = offsets_of(counts)
    dx = api.grouped_mxfp4_gemm(a, sa, off.to(DEV), wt, st, out_dtype=torch.float32)
    want, mag = ref.product(a.cpu(), sa.cpu(), off, wt.cpu(), st.cpu())
    near(dx.cpu(), want, mag, N, torch.float32)
    back = api.mxfp4_values(wt, st, dtype=torch.float32, weights=True).transpose(1, 2)
    # E2M1's steps are at most a fifth of a block's largest magnitude up to
    # twice the clipped part (6 of less than 8): within a third of it
    top = w.abs().amax()
    assert (back - w).abs().max() <= top / 3


# ------------------------------------------------- quick succession, graphs, threads

def batch(seed):
    """A call of each kernel: few, some and many rows an expert, and the movement."""
    calls = []
    for counts, K, N in (([8], 128, 256), ([300], 256, 144), ([60, 61], 640, 128), ([0, 5, 700, 3], 96, 272), ([2] * 30, 512, 512)):
        R, a, sa, off, w, sw = product_case(counts, 0, 0, K, N, seed=seed + K)
        args = [t.to(DEV) for t in (a, sa, off, w, sw)]
        calls.append(lambda args=args: (api.grouped_mxfp4_gemm(*args),))
    for T, E, k, d in ((40, 16, 3, 96), (1500, 40, 4, 64)):
        x, idx, w = normal(T, d, seed=seed).to(DEV), routes(T, E, k, 0.0, seed=seed).to(DEV), torch.rand(T, k, generator=gen(seed)).to(DEV)
        calls.append(lambda x=x, idx=idx, E=E: api.dispatch(x, idx, E, "floor"))
        calls.append(lambda x=x, idx=idx, E=E, w=w: move(x, idx, E, w))
    gu = normal(77, 192, seed=seed).to(DEV)
    calls.append(lambda: tuple(api.swiglu_mxfp4(gu[:, :96], gu[:, 96:], want_h=True)))
    return calls


def move(x, idx, E, w):
    r = api.dispatch(x, idx, E)
    out = api.combine(r.rows, r.inv_row, w)
    g = api.combine_backward(out, r.rows, r.inv_row, w)
    return r.rows, r.inv_row, out, g.dy, g.dw, api.dispatch_backward(g.dy, r.inv_row)


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


def test_calls_in_quick_succession():
    calls = batch(1)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[c() for c in calls] for _ in range(20)]
        assert all(same(p, q) for row in got for p, q in zip(row, want))


def test_captured_graphs_replay_on_new_inputs():
    # two graphs of the same operators that share a workspace, replayed in
    # turn on inputs written after the capture
    T, E, k, d, N = 1200, 24, 3, 128, 160
    assert api.moe_dispatch_workspace_size(T, E, k) > 0
    ws = torch.empty(api.moe_dispatch_workspace_size(T, E, k), dtype=torch.uint8, device=DEV)
    w, sw = (t.to(DEV) for t in weights(E, N, d, 1))

    def step(x, idx):
        r = api.dispatch(x, idx, E, quantize="fit", workspace=ws)
        y = api.grouped_mxfp4_gemm(r.rows, r.scales, r.offsets, w, sw)
        out = api.combine(y, r.inv_row)
        return out, api.combine_backward(out, y, r.inv_row, want_dw=True).dw

    inputs = [(normal(T, d, seed=s).to(DEV), routes(T, E, k, 0.0, seed=s).to(DEV)) for s in range(4)]
    want = [step(*i) for i in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for s in range(2):
            x, idx = (t.clone() for t in inputs[s])
            step(x, idx)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = step(x, idx)
            graphs.append((g, x, idx, out))
        for n in range(12):
            g, x, idx, out = graphs[n % 2]
            i = (n * 5 + n // 4) % 4
            x.copy_(inputs[i][0])
            idx.copy_(inputs[i][1])
            g.replay()
            got = [t.clone() for t in out]
            assert same(got, want[i]), n
    torch.cuda.current_stream().wait_stream(side)


def test_calls_from_two_threads():
    errors, start = [], threading.Barrier(2)

    def work(seed):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                calls = batch(seed)
                want = [c() for c in calls]
                stream.synchronize()
                start.wait(timeout=60)
                for _ in range(60):
                    got = [c() for c in calls]
                    assert all(same(p, q) for p, q in zip(got, want))
        except Exception as e:  # (an assertion in a thread would be lost)
            errors.append(repr(e))
            start.abort()

    threads = [threading.Thread(target=work, args=(s,), daemon=True) for s in (3, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errors and not any(t.is_alive() for t in threads)


def test_calls_on_a_given_stream():
    T, E, k, d = 1500, 24, 3, 96
    x, idx, w = normal(T, d, seed=1).to(DEV), routes(T, E, k, 0.0, seed=1).to(DEV), torch.rand(T, k, generator=gen(2)).to(DEV)
    for mx in (None, "floor"):
        check_on_stream(lambda t, **kw: api.dispatch(t[0], t[1], E, mx, **kw), [x, idx])
    r = api.dispatch(x, idx, E)
    check_on_stream(lambda t, **kw: api.combine(t[0], t[1], t[2], t[3], **kw), [r.rows, r.inv_row, w, x])
    check_on_stream(lambda t, **kw: api.dispatch_backward(t[0], t[1], **kw), [r.rows, r.inv_row])
    check_on_stream(lambda t, **kw: api.combine_backward(*t, **kw), [x, r.rows, r.inv_row, w])
    three = normal(32, 48, 64, seed=3).to(DEV)
    check_on_stream(lambda t, **kw: api.quantize_mxfp4(t[0].transpose(0, 1), weights=True, **kw), [three])
    q = api.quantize_mxfp4(x)
    check_on_stream(lambda t, **kw: api.mxfp4_values(t[0], t[1], **kw), list(q))
    check_on_stream(lambda t, **kw: api.swiglu_mxfp4(t[0][:, :32], t[0][:, 32:64], want_h=True, **kw), [x])
    for counts in ([50, 0, 20], [500, 10]):
        R, a, sa, off, wc, sw = product_case(counts, 0, 0, 256, 128, seed=4)
        check_on_stream(lambda t, **kw: api.grouped_mxfp4_gemm(*t, **kw), [v.to(DEV) for v in (a, sa, off, wc, sw)])


# ------------------------------------------------------- past 2^31 elements

def test_quantize_and_values_past_32_bits():
    x, e = tall((1 << 20) + 77, 2080, 1)
    assert x.numel() > 1 << 31
    codes, scales = api.quantize_mxfp4(x)
    c, s = api.quantize_mxfp4(e)
    assert torch.equal(ends_of(codes), c) and torch.equal(ends_of(scales), s) and not codes[ENDS:-ENDS].any()
    v = api.mxfp4_values(codes, scales)
    assert torch.equal(ends_of(v), api.mxfp4_values(c, s)) and not v[ENDS:-ENDS].any()


def test_weights_past_32_bits():
    E, N, K = 40, 8208, 6560
    assert E * N * K > 1 << 31
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[0], w[-1] = normal(N, K, seed=1).to(DEV), normal(N, K, seed=2).to(DEV)
    codes, scales = api.quantize_mxfp4(w, weights=True)
    ends = torch.stack([w[0], w[-1]])
    c, s = api.quantize_mxfp4(ends, weights=True)
    assert torch.equal(codes[[0, -1]], c) and torch.equal(scales[[0, -1]], s)
    assert torch.equal(api.mxfp4_values(codes, scales, weights=True)[-1], api.mxfp4_values(c, s, weights=True)[-1])


def test_swiglu_past_32_bits():
    f = 2080
    gu, e = tall((1 << 20) + 77, 2 * f, 2)
    r, w = (api.swiglu_mxfp4(t[:, :f], t[:, f:], want_h=True) for t in (gu, e))
    assert r.h.numel() > 1 << 31
    assert torch.equal(ends_of(r.h), w.h) and torch.equal(ends_of(r.codes), w.codes) and torch.equal(ends_of(r.scales), w.scales)


def test_movement_past_32_bits():
    T, k, d, E = 140_000, 8, 2048, 16
    assert T * k * d > 1 << 31
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    e = normal(2 * ENDS, d, seed=3).to(DEV)
    x[:ENDS], x[T - ENDS:] = e[:ENDS], e[ENDS:]
    idx = torch.full((T, k), 5, dtype=torch.int32, device=DEV)  # all in one expert: rows in token order
    r = api.dispatch(x, idx, E)
    want = e.repeat_interleave(k, 0)
    assert torch.equal(r.rows[:ENDS * k], want[:ENDS * k]) and torch.equal(r.rows[-ENDS * k:], want[ENDS * k:])
    assert torch.equal(r.inv_row.flatten(), torch.arange(T * k, device=DEV, dtype=torch.int32))
    mx = api.dispatch(x, idx, E, "floor")
    c, s = api.quantize_mxfp4(want)
    assert torch.equal(mx.rows[-ENDS * k:], c[ENDS * k:]) and torch.equal(mx.scales[-ENDS * k:], s[ENDS * k:])
    w = torch.rand(T, k, generator=gen(4)).to(DEV)
    out = api.combine(r.rows, r.inv_row, w)
    ends = torch.cat([w[:ENDS], w[-ENDS:]])
    small = torch.arange(2 * ENDS * k, device=DEV, dtype=torch.int32).view(-1, k)
    assert torch.equal(ends_of(out), api.combine(want, small, ends))
    g, h = api.combine_backward(x, r.rows, r.inv_row, w), api.combine_backward(e, want, small, ends)
    # (few tokens are summed in another order; every term is a square, so that
    # the terms' magnitudes add up to the sum)
    assert ((ends_of(g.dw) - h.dw).abs() <= 2 * (d // 32 + 20) * U * h.dw).all()
    assert torch.equal(g.dy[-ENDS * k:], h.dy[ENDS * k:])


@pytest.mark.parametrize("E,R,K,N", [(3, 300_032, 128, 7168), (200, 8_200, 32, 262_400), (1024, 49_100, 32, 44_032)],
                         ids=["many", "some", "few"])
def test_product_past_32_bits(E, R, K, N):
    assert R * N > 1 << 31
    x, e = tall(R, K, 3)
    a, sa = api.quantize_mxfp4(x)
    w, sw = weights(4, N, K, 4)
    w, sw = (t.repeat(E // 4 + 1, 1, 1)[:E].contiguous() for t in (w, sw))
    off = torch.linspace(0, R, E + 1).round().to(torch.int32)
    out = api.grouped_mxfp4_gemm(a, sa, off.to(DEV), w.to(DEV), sw.to(DEV))
    first, last = int((off[1:] <= 0).sum()), E - 1
    for rows, g in ((slice(0, min(ENDS, int(off[first + 1]))), first), (slice(max(R - ENDS, int(off[last])), R), last)):
        n = rows.stop - rows.start
        y, mag = ref.product(a[rows].cpu(), sa[rows].cpu(), offsets_of([n]), w[g:g + 1], sw[g:g + 1])
        near(out[rows].cpu(), y, mag, K, torch.bfloat16)


# --------------------------------------------------------------- long launches

SHORT_LIMIT = """
import torch
from routed_expert_ffn_gemm_gb300 import api
def full(v, *s):
    return torch.full(s, v, dtype=torch.uint8, device="cuda")
for R, E, K, N in ((16384, 2, 4096, 14336), (8192, 100, 4096, 14336), (256, 256, 2048, 14336)):
    off = torch.linspace(0, R, E + 1).to(torch.int32).cuda()
    y = api.grouped_mxfp4_gemm(full(0x22, R, K // 2), full(127, R, K // 32), off, full(0x22, E, N, K // 2), full(127, E, K // 32, N))
    assert (y == K).all(), (R, E, K, N)
assert api.moe_read_device_status() == api.OK
print("complete")
"""


def test_long_products_are_not_cut_off():
    # launches of 0.3 to 1 ms under a limit of 0.05 ms for stuck ones: what the
    # limit leaves a launch grows with its work
    r = subprocess.run([sys.executable, "-c", SHORT_LIMIT], cwd=ROOT, env=dict(os.environ, MOE_WAIT_LIMIT_NS="50000"),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "complete" in r.stdout, r.stdout + r.stderr
