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
