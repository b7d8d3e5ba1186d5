"""The norm's and the 4-bit calls from eight host threads at once, each on its own
stream, in a fresh process (the library's first use of each kernel is concurrent
too): every thread's results equal the single-threaded ones bit for bit."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
from fp8_block_scaled_11_b200 import build, inputs, ops

build.build()
torch.cuda.init()
x = inputs.random_matrix(600, 2048, seed=71, dtype=torch.bfloat16).cuda()
r = inputs.random_matrix(600, 2048, seed=72, dtype=torch.bfloat16).cuda()
w = inputs.random_matrix(1, 2048, seed=73, dtype=torch.float32).cuda()[0]
W = inputs.random_matrix(1100, 2048, seed=74, dtype=torch.bfloat16).cuda()
big = inputs.random_matrix(6000, 2048, seed=75, dtype=torch.bfloat16).cuda()
torch.cuda.synchronize()

def work():
    out = []
    wq, ws = ops.fp4_quant_1x32(W)
    bq, bs = ops.fp4_quant_1x32(big)
    for m in (1, 20, 50, 600):
        q, s, h, rstd, _ = ops.fp4_rmsnorm_quant_1x32(x[:m], w, r[:m])
        out += [q, rstd, h, ops.fp4_scaled_gemm(q, wq, s, ws)]
    out.append(ops.fp4_scaled_gemm(bq, wq, bs, ws, out_dtype=torch.float32))       # CTA pairs
    out.append(ops.fp4_scaled_gemm(bq, bq, bs, bs))
    q8, s8, h, rstd, y = ops.fp8_rmsnorm_quant_1x128(x, w, r, want_y=True)
    out += [q8, s8, y]
    out += list(ops.fp8bs_rmsnorm_backward(y, h, w, rstd, dh=r))
    qt, st = ops.fp4_quant_1x32(x[:576], transpose_out=True)
    out += [qt, ops.fp4_dequant_1x32(qt, st)]
    return out

results, errors = [None] * 8, []
start = threading.Barrier(8)

def thread(i):
    try:
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            out = [work() for _ in range(2)][1]
        stream.synchronize()
        results[i] = [t.cpu() for t in out]
    except Exception as e:           # reported below
        errors.append(repr(e))

ts = [threading.Thread(target=thread, args=(i,)) for i in range(8)]
for t in ts: t.start()
for t in ts: t.join()
assert not errors, errors
assert ops.fp8bs_check_device_error() == 0
ref = [t.cpu() for t in work()]
torch.cuda.synchronize()
for res in results:
    for a, b in zip(res, ref):
        assert torch.equal(a.contiguous(), b.contiguous())
print("threads ok")
'''


def test_eight_threads_and_streams():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "threads ok" in r.stdout


@pytest.mark.parametrize("M", [1, 40, 300, 2300])
def test_chain_without_waits(M):
    """Sixty steps of dependent calls over the same buffers, each written again as soon as the call that reads it is
    launched: the same bits with the host waiting after every call, without waiting, and from a replayed graph."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from fp8_block_scaled_11_b200 import build, inputs, ops
    build.build()
    K = 1024
    x0 = inputs.random_matrix(M, K, seed=81).cuda()
    wq, ws = ops.fp4_quant_1x32(inputs.random_matrix(K, K, seed=82, scale=K ** -0.5).cuda())
    g = torch.linspace(0.5, 1.5, K, device="cuda").bfloat16()
    x, r = torch.empty_like(x0), torch.empty_like(x0)
    out4, out8 = ops.rmsnorm_quant_buffers(x0, residual=True, bits=4), ops.rmsnorm_quant_buffers(x0, want_y=True)
    q, s = ops.fp4_quant_1x32(x0)
    dx, dw = torch.empty_like(x0), torch.empty(K, device="cuda")
    total = torch.empty(K, device="cuda")
    bwd = ops.rmsnorm_backward_workspace(x0)

    def steps(wait):
        x.copy_(x0)
        r.copy_(x0)
        total.zero_()
        for _ in range(60):
            _, _, h, rstd, _ = ops.fp4_rmsnorm_quant_1x32(x, g, residual=r, out=out4)
            wait()
            ops.fp4_scaled_gemm(out4[0], wq, out4[1], ws, out=x)
            wait()
            ops.fp4_quant_1x32(x, q=q, scale=s)
            wait()
            ops.fp4_dequant_1x32(q, s, out=r)
            wait()
            y = ops.fp8_rmsnorm_quant_1x128(r, g, out=out8)[4]
            wait()
            ops.fp8bs_rmsnorm_backward(y, h, g, rstd, dh=x, out=(dx, dw), workspace=bwd)
            wait()
            total.add_(dw)
            r.add_(dx, alpha=0.5)
            wait()
        return [t.clone() for t in (x, r, total, out8[0], dx)]

    want = steps(torch.cuda.synchronize)
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    got = steps(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = steps(lambda: None)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


FIRST = r'''
import sys
sys.path.insert(0, sys.argv[1])
import torch
from fp8_block_scaled_11_b200 import build, inputs, ops

build.build()
x = inputs.random_matrix(600, 1024, seed=91).cuda()
w = torch.ones(1024, device="cuda").bfloat16()

def calls():
    out = []
    for m in (1, 600):
        q, s, h, rstd, y = ops.fp4_rmsnorm_quant_1x32(x[:m], w, x[:m], want_y=True)
        wq, ws = ops.fp4_quant_1x32(x)
        out += [q, ops.fp4_scaled_gemm(q, wq, s, ws), *ops.fp8bs_rmsnorm_backward(y, h, w, rstd)]
    big = torch.cat([x] * 8)
    bq, bs = ops.fp4_quant_1x32(big)
    return out + [ops.fp4_scaled_gemm(bq, bq, bs, bs)]           # CTA pairs

torch.cuda.synchronize()
side = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):
    got = calls()
g.replay()
torch.cuda.synchronize()
assert ops.fp8bs_check_device_error() == 0
for a, b in zip(got, calls()):
    assert torch.equal(a, b)
print("captured ok")
'''


def test_first_calls_inside_a_capture():
    """The library's very first use of each kernel may be inside a graph's capture."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stderr[-2000:]
