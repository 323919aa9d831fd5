"""The expert-training operators launched in other ways than one call at a
time on the current stream: in quick succession, on given streams, from
several threads, on results past 2^31 elements."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from routed_expert_ffn_gemm_gb300 import api, build, inputs
from tests import train_reference as ref
from tests.test_gpu_expert_training import close, gemm_case, gen, normal, offsets_of, routed

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()
    api._lib()
    yield
    assert api.moe_read_device_status() == api.OK


def test_products_in_quick_succession():
    # launches of one unit each, few rows, many rows and weight gradients in
    # turn: each takes over shared memory and barriers that the one before
    # has just left
    cases = []
    for counts, K, N, transposed in (([8], 128, 256, False), ([300], 128, 256, False), ([300], 272, 256, True),
                                     ([40], 640, 128, True), ([90, 1], 256, 256, False)):
        R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, transposed, seed=K)
        args = [t.to(DEV) for t in (a, sa, off, w, sw)]
        cases.append(lambda args=args, t=transposed: api.grouped_block_gemm(*args, t))
    for rows, kind in ((5, "pow2"), (70, None)):
        dy, x, xs, off = normal(rows, 256, seed=1).to(DEV), normal(rows, 256, seed=2), None, offsets_of([rows]).to(DEV)
        if kind:
            x, xs = ref.quantize(x, kind)
            xs = xs.to(DEV)
        x = x.to(DEV)
        cases.append(lambda dy=dy, x=x, xs=xs, off=off: api.grouped_wgrad(dy, x, xs, off))
    want = [c() for c in cases]
    got = [[c() for c in cases] for _ in range(300)]
    for row in got:
        assert all(torch.equal(p, q) for p, q in zip(row, want))


@pytest.mark.parametrize("E,k", [(2, 1), (8, 2), (40, 4), (256, 8), (1000, 8)])
def test_router_sum_with_idle_ctas(E, k):
    # with few experts most CTAs of the sum's cluster have nothing to add and
    # hand their share over at once
    T = 3000
    logits, idx, _ = routed(T, E, k, seed=E)
    want = ref.router(logits.double(), idx, None, 0.3, 0.02)
    logits, idx = logits.to(DEV), idx.to(DEV)
    runs = [api.router_losses(logits, idx, 0.3, 0.02) for _ in range(200)]
    close(runs[0].loss, torch.stack(want[:2]))
    assert torch.equal(runs[0].counts.cpu(), want[2])
    for r in runs:
        assert torch.equal(r.loss, runs[0].loss) and torch.equal(r.counts, runs[0].counts)


def test_router_losses_from_two_threads():
    # both sizes run the same kernel, with 52 800 and 67 584 bytes of shared
    # memory: a call's launch must not depend on another thread's calls
    T, k, errors = 200, 4, []

    def work(E):
        try:
            logits, idx, _ = routed(T, E, k, seed=E)
            want = ref.router(logits.double(), idx, None, 0.3, 0.02)
            logits, idx = logits.to(DEV), idx.to(DEV)
            r = api.router_losses(logits, idx, 0.3, 0.02)
            ws = torch.empty(api.moe_router_losses_workspace_size(T, E), dtype=torch.uint8, device=DEV)
            args = (T, E, k, logits.data_ptr(), idx.data_ptr(), None, 0.3, 0.02, r.loss.data_ptr(), r.counts.data_ptr(),
                    r.lse.data_ptr(), ws.data_ptr(), ws.numel(), api._stream(None))
            start.wait(timeout=60)
            for _ in range(20000):
                api._call("moe_router_losses", *args)
            torch.cuda.synchronize()
            close(r.loss, torch.stack(want[:2]))
        except Exception as e:  # (an assertion in a thread would be lost)
            errors.append(f"E = {E}: {e!r}")
            start.abort()

    start = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=(E,), daemon=True) for E in (400, 512)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errors and not any(t.is_alive() for t in threads)


# What a call with stream= reads is made on that stream behind some 50 ms of
# waiting, and the current stream meanwhile fills every freed block with other
# values: a copy, a buffer or a launch on the current stream shows.

def values_of(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)]


def check_on_stream(fn, tensors):
    """fn(tensors, **kw) with stream=side against the same call without."""
    want = [t.clone() for t in values_of(fn(tensors))]
    sizes = sorted({t.numel() * t.element_size() for t in want} | {1 << p for p in range(9, 22)})
    later = [None if t is None else torch.zeros_like(t) for t in tensors]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        for t, v in zip(later, tensors):
            if t is not None:
                t.copy_(v)
    got = fn(later, stream=side)
    churn = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(8)]
    del churn
    side.synchronize()
    got = values_of(got)
    assert len(got) == len(want) and all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("shape,axes", [((300, 256), None), ((40, 30, 384), (1, 0, 2)), ((96, 128, 5), (2, 0, 1))])
def test_quantize_blocks_on_a_given_stream(shape, axes):
    x = normal(*shape, seed=3).to(DEV)
    check_on_stream(lambda t, **kw: api.quantize_blocks(t[0] if axes is None else t[0].permute(axes), "pow2", **kw), [x])


def test_products_and_gradients_on_a_given_stream():
    counts, K, N = [50, 0, 120], 256, 384
    R, a, sa, off, w, sw = gemm_case(counts, 0, 0, K, N, False, seed=6)
    a, sa, off, w, sw = (t.to(DEV) for t in (a, sa, off, w, sw))
    check_on_stream(lambda t, **kw: api.grouped_block_gemm(*t, **kw), [a, sa, off, w, sw])
    dy = normal(R, N, seed=7).to(DEV)
    check_on_stream(lambda t, **kw: api.grouped_wgrad(*t, **kw), [dy, a, sa, off])
    check_on_stream(lambda t, **kw: api.grouped_wgrad(t[0], t[1], None, t[2], t[3].clone() if not kw else t[3], True, **kw),
                    [dy, normal(R, K, seed=8).to(DEV), off, torch.ones(3, N, K, device=DEV)])


def test_swiglu_on_a_given_stream():
    gu, dh = normal(333, 512, seed=9).to(DEV), normal(333, 256, seed=10).to(DEV)
    check_on_stream(lambda t, **kw: api.swiglu_save(t[0][:, :256], t[0][:, 256:], want_h=True, **kw), [gu])
    saved, scales = api.quantize_blocks(gu.view(333, 2, 256).transpose(0, 1), "pow2")
    check_on_stream(lambda t, **kw: api.swiglu_backward(*t, want_h=True, want_codes=True, **kw), [saved, scales, dh])


@pytest.mark.parametrize("T,E,k", [(64, 8, 2), (5000, 60, 4)])
def test_router_on_a_given_stream(T, E, k):
    # (the workspace that the call makes for itself among what must not be reused)
    logits, idx, w = (t.to(DEV) for t in routed(T, E, k, seed=1))
    check_on_stream(lambda t, **kw: tuple(api.router_losses(t[0], t[1], 0.3, 0.02, **kw))[:3], [logits, idx])
    r = api.router_losses(logits, idx, 0.3, 0.02)
    check_on_stream(lambda t, **kw: api.router_losses_backward(
        t[0], t[1], api.RouterLosses(t[2], t[3], t[4], 0.3, 0.02), topk_w=t[5], d_topk_w=t[5], **kw),
        [logits, idx, r.loss, r.counts, r.lse, w])


@pytest.mark.parametrize("wfmt", ["bf16", "fp8"])
def test_layer_forward_on_a_given_stream(wfmt):
    shape = inputs.MoEShape("stream", T=40, d=256, ffn=384, E=8, k=2, ffn_shared=256, wfmt=wfmt)
    case = inputs.make_case(shape, seed=4, device=DEV)
    names = sorted(case, key=str)
    names = [n for n in names if isinstance(case[n], torch.Tensor)]
    check_on_stream(lambda t, **kw: api.layer_forward(api.problem_of(shape), dict(case, **dict(zip(names, t))),
                                                      want_routing=True, **kw), [case[n] for n in names])


# Results past 2^31 elements: the first and the last rows against the same
# rows by themselves (what lies between is zero).

ENDS = 40


def ends_of(t, dim=0):
    return torch.cat([t.narrow(dim, 0, ENDS), t.narrow(dim, t.shape[dim] - ENDS, ENDS)], dim)


def tall(rows, cols, seed, dtype=torch.bfloat16):
    x = torch.zeros(rows, cols, dtype=dtype, device=DEV)
    e = normal(2 * ENDS, cols, seed=seed).to(dtype).to(DEV)
    x[:ENDS], x[rows - ENDS:] = e[:ENDS], e[ENDS:]
    return x, e


def test_quantize_blocks_past_32_bits():
    x, e = tall((1 << 20) + 77, 2056, 1)
    assert x.numel() > 1 << 31
    codes, scales = api.quantize_blocks(x, "pow2")
    c, s = api.quantize_blocks(e, "pow2")
    assert torch.equal(ends_of(codes), c) and torch.equal(ends_of(scales), s)
    assert not codes[ENDS:-ENDS].any()


def test_swiglu_past_32_bits():
    f = 2064
    gu, e = tall((1 << 20) + 77, 2 * f, 2)
    r, w = (api.swiglu_save(t[:, :f], t[:, f:], want_h=True) for t in (gu, e))
    assert r.h.numel() > 1 << 31
    assert torch.equal(ends_of(r.h), w.h) and torch.equal(ends_of(r.codes), w.codes)
    assert torch.equal(ends_of(r.saved, 1), w.saved) and torch.equal(ends_of(r.saved_scales, 1), w.saved_scales)
    del gu
    d, v = (api.swiglu_backward(t.saved, t.saved_scales, t.h, want_h=True) for t in (r, w))
    assert torch.equal(ends_of(d.d_gu), v.d_gu) and torch.equal(ends_of(d.h), v.h)


@pytest.mark.parametrize("E,R,K,N", [(3, 300_032, 128, 7168), (1024, 49_100, 16, 44_032)], ids=["many", "few"])
def test_block_gemm_past_32_bits(E, R, K, N):
    assert R * N > 1 << 31
    x, e = tall(R, K, 3)
    a, sa = api.quantize_blocks(x)
    w, sw = ref.quantize(normal(8, N, K, seed=4), "amax")
    w = w.repeat(E // 8 + 1, 1, 1)[:E].contiguous()
    sw = torch.rand(E, -(-N // 128), 1, generator=gen(5)) + 0.5
    off = torch.linspace(0, R, E + 1).round().to(torch.int32)
    out = api.grouped_block_gemm(a, sa, off.to(DEV), w.to(DEV), sw.to(DEV))
    first, last = int((off[1:] <= 0).sum()), E - 1
    for rows, g in ((slice(0, min(ENDS, int(off[first + 1]))), first), (slice(max(R - ENDS, int(off[last])), R), last)):
        n = rows.stop - rows.start
        y, mag = ref.block_gemm(a[rows].cpu(), sa[rows].cpu(), offsets_of([n]), w[g:g + 1], sw[g:g + 1], False)
        # (as the block product's tests have it, for one block)
        assert ((out[rows].cpu().double() - y).abs() <= 36 * 2.0 ** -24 * mag + 2.0 ** -8 * y.abs()).all()


def test_wgrad_past_32_bits():
    E, N, K = 64, 8192, 4112
    assert E * N * K > 1 << 31
    counts = [5] + [0] * (E - 2) + [21]
    dy, x = normal(26, N, seed=6).to(DEV), normal(26, K, seed=7).to(DEV)
    dw = torch.full((E, N, K), 7.0, device=DEV)
    api.grouped_wgrad(dy, x, None, offsets_of(counts).to(DEV), dw)
    for g, rows in ((0, slice(0, 5)), (E - 1, slice(5, 26))):
        n = rows.stop - rows.start
        assert torch.equal(dw[g], api.grouped_wgrad(dy[rows], x[rows], None, offsets_of([n]).to(DEV))[0])
    assert not any(dw[g].any() for g in range(1, E - 1))


SHORT_LIMIT = """
import torch
from routed_expert_ffn_gemm_gb300 import api
def codes(*s):
    return torch.full(s, 0x38, dtype=torch.uint8, device="cuda")  # 1.0
def ones(*s):
    return torch.ones(*s, device="cuda")
for R, E, K, N, t in ((8192, 2, 4096, 14336, False), (8192, 2, 4096, 14336, True), (4096, 64, 4096, 7168, False),
                      (256, 128, 2048, 7168, False)):
    off = torch.linspace(0, R, E + 1).to(torch.int32).cuda()
    w, sw = ((K, N), (K // 128, N // 128)) if t else ((N, K), (N // 128, K // 128))
    y = api.grouped_block_gemm(codes(R, K), ones(R, K // 128), off, codes(E, *w), ones(E, *sw), t)
    assert (y == K).all(), (R, E, K, N, t)
R, E, N, K = 8192, 2, 4096, 14336
off = torch.tensor([0, 4096, 8192], dtype=torch.int32, device="cuda")
dy = torch.ones(R, N, dtype=torch.bfloat16, device="cuda")
dw = api.grouped_wgrad(dy, codes(R, K), ones(R, K // 128), off)
assert (dw == 4096).all()
assert api.moe_read_device_status() == api.OK
print("complete")
"""


def test_long_products_are_not_cut_off():
    # launches of 0.2 to 1 ms under a limit of 0.05 ms for stuck ones: what
    # the limit leaves a launch grows with its work
    r = subprocess.run([sys.executable, "-c", SHORT_LIMIT], cwd=ROOT, env=dict(os.environ, MOE_WAIT_LIMIT_NS="50000"),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "complete" in r.stdout, r.stdout + r.stderr
