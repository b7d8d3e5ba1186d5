"""Argument checks of the norm's and the 4-bit entry points (no GPU: every call
fails validation before anything is launched), and the Python binding's own."""
import ctypes
import os
import re

import pytest
import torch

from fp8_block_scaled_11_b200 import build, ops

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4
GOOD, BAD = 0x10000, 0x10008
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


def test_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8bs.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp4_\w+)\s*\(", text))
    assert names == {"fp4_rmsnorm_quant_1x32", "fp4_scale_tiles_size", "fp4_quant_1x32", "fp4_dequant_1x32",
                     "fp4_scaled_gemm", "fp4_scaled_gemm_workspace_size"}
    for n in names:
        assert hasattr(L, n)


def norm8(L, x=GOOD, ldx=256, r=GOOD, ldr=256, xt=0, rows=4, cols=256, w=GOOD, wt=0, eps=1e-6, h=GOOD, ldh=256,
          rstd=GOOD, y=0, ldy=0, q=GOOD, ldq=256, s=GOOD, lds=4, rule=0):
    return L.fp8_rmsnorm_quant_1x128(x, ldx, r, ldr, xt, rows, cols, w, wt, ctypes.c_float(eps), h, ldh, rstd, y, ldy,
                                     q, ldq, s, lds, rule, None)


def norm4(L, cols=256, ldq=128, **kw):
    a = dict(x=GOOD, ldx=256, r=0, ldr=0, xt=0, rows=4, w=GOOD, wt=1, eps=0.0, h=0, ldh=0, rstd=0, y=0, ldy=0, q=GOOD,
             s=GOOD)
    a.update(kw)
    return L.fp4_rmsnorm_quant_1x32(a["x"], a["ldx"], a["r"], a["ldr"], a["xt"], a["rows"], cols, a["w"], a["wt"],
                                    ctypes.c_float(a["eps"]), a["h"], a["ldh"], a["rstd"], a["y"], a["ldy"], a["q"],
                                    ldq, a["s"], None)


def test_norm_validation(L):
    for kw in ({"x": 0}, {"w": 0}, {"q": 0}, {"s": 0}, {"rows": 0}, {"cols": 0}, {"h": 0}, {"r": 0},
               {"ldx": 240}, {"ldr": 240}, {"ldh": 240}, {"ldq": 240}, {"lds": 0}, {"y": GOOD, "ldy": 240},
               {"eps": -1.0}, {"eps": float("nan")}, {"rows": 1 << 31, "lds": 1 << 31}):
        assert norm8(L, **kw) == INVALID, kw
    for kw in ({"xt": 2}, {"wt": 7}, {"rule": 5}):
        assert norm8(L, **kw) == UNSUPPORTED, kw
    for kw in ({"x": BAD}, {"r": BAD}, {"w": BAD}, {"h": BAD}, {"q": BAD}, {"s": BAD}, {"y": BAD, "ldy": 256},
               {"rstd": GOOD + 2}, {"ldx": 260}, {"ldr": 260}, {"ldh": 260}, {"ldq": 264}, {"lds": 6},
               {"cols": 200}, {"y": GOOD, "ldy": 260}):
        assert norm8(L, **kw) == ALIGN, kw
    assert norm4(L, cols=240) == ALIGN                # 4 bits: cols % 32
    assert norm4(L, ldq=112) == INVALID
    assert norm4(L, ldq=136) == ALIGN
    assert norm4(L, s=BAD) == ALIGN
    assert norm4(L, s=0) == INVALID


def test_backward_validation(L):
    def back(dy=GOOD, lddy=256, h=GOOD, ldh=256, dh=GOOD, lddh=256, xt=0, rows=4, cols=256, w=GOOD, wt=0, rstd=GOOD,
             dx=GOOD, lddx=256, dw=GOOD, ws=0, wsb=0):
        return L.fp8bs_rmsnorm_backward(dy, lddy, h, ldh, dh, lddh, xt, rows, cols, w, wt, rstd, dx, lddx, dw, ws, wsb,
                                        None)
    for kw in ({"dy": 0}, {"h": 0}, {"w": 0}, {"rstd": 0}, {"dx": 0}, {"dw": 0}, {"rows": 0}, {"cols": 0},
               {"lddy": 128}, {"ldh": 128}, {"lddh": 128}, {"lddx": 128}):
        assert back(**kw) == INVALID, kw
    for kw in ({"dy": BAD}, {"h": BAD}, {"dh": BAD}, {"w": BAD}, {"dx": BAD}, {"rstd": GOOD + 1}, {"dw": GOOD + 2},
               {"lddy": 260}, {"ldh": 260}, {"lddh": 260}, {"lddx": 260}, {"cols": 200}):
        assert back(**kw) == ALIGN, kw
    assert back(xt=3) == UNSUPPORTED and back(wt=-1) == UNSUPPORTED
    assert L.fp8bs_rmsnorm_backward_workspace_size(0, 16) == 0
    # one row of partial sums per row of a small batch; wide rows: the rows' means too
    assert L.fp8bs_rmsnorm_backward_workspace_size(1, 256) >= 256 * 4
    assert L.fp8bs_rmsnorm_backward_workspace_size(16640, 8192) < 64 << 20


def test_quant_validation(L):
    def quant(x=GOOD, xt=0, rows=64, cols=256, ldx=256, q=GOOD, ldq=128, s=GOOD, t=0):
        return L.fp4_quant_1x32(x, xt, rows, cols, ldx, q, ldq, s, t, None)
    for kw in ({"x": 0}, {"q": 0}, {"s": 0}, {"rows": 0}, {"cols": 0}, {"ldx": 240}, {"ldq": 112}, {"t": 2},
               {"t": 1, "ldq": 16}):
        assert quant(**kw) == INVALID, kw
    for kw in ({"x": BAD}, {"q": BAD}, {"s": BAD}, {"ldx": 260}, {"ldq": 136}, {"cols": 240}, {"rows": 48, "t": 1},
               {"cols": 248, "t": 1}):
        assert quant(**kw) == ALIGN, kw
    assert quant(xt=2) == UNSUPPORTED
    assert L.fp4_scale_tiles_size(129, 160) == 2 * 2 * 512 and L.fp4_scale_tiles_size(0, 1) == 0

    def deq(q=GOOD, ldq=128, s=GOOD, rows=8, cols=256, o=GOOD, ot=0, ldo=256):
        return L.fp4_dequant_1x32(q, ldq, s, rows, cols, o, ot, ldo, None)
    for kw in ({"q": 0}, {"s": 0}, {"o": 0}, {"rows": 0}, {"ldq": 112}, {"ldo": 240}):
        assert deq(**kw) == INVALID, kw
    for kw in ({"q": BAD}, {"s": BAD}, {"o": BAD}, {"cols": 240}, {"ldo": 260}, {"ldq": 136}):
        assert deq(**kw) == ALIGN, kw
    assert deq(ot=4) == UNSUPPORTED


def test_product_validation(L):
    def mm(M=64, N=64, K=256, A=GOOD, lda=128, B=GOOD, ldb=128, sa=GOOD, sb=GOOD, D=GOOD, ldd=64, od=0, ws=0, wsb=0):
        return L.fp4_scaled_gemm(M, N, K, A, lda, B, ldb, sa, sb, D, ldd, od, ws, wsb, None)
    for kw in ({"A": 0}, {"B": 0}, {"sa": 0}, {"sb": 0}, {"D": 0}, {"M": 0}, {"N": 0}, {"K": 16}, {"lda": 112},
               {"ldb": 112}, {"ldd": 63}, {"M": 1 << 31}):
        assert mm(**kw) == INVALID, kw
    for kw in ({"A": BAD}, {"B": BAD}, {"sa": BAD}, {"sb": BAD}, {"D": GOOD + 1}, {"D": GOOD + 2, "od": 1}, {"K": 240},
               {"lda": 136}, {"ldb": 136}):
        assert mm(**kw) == ALIGN, kw
    assert mm(od=2) == UNSUPPORTED
    assert L.fp4_scaled_gemm_workspace_size(16640, 5120, 8192) == 0
    # one token's K is shared by a cluster; very long K over one tile goes through the workspace
    assert L.fp4_scaled_gemm_workspace_size(1, 5120, 8192) == 0
    n = L.fp4_scaled_gemm_workspace_size(16, 130, 131072)
    assert n > 0 and n % (16 * 132 * 4) == 0


def test_binding_refuses():
    """Shapes, dtypes and layouts are refused before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w, torch.zeros(4, 32, dtype=torch.bfloat16))      # residual's shape
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w, torch.zeros(4, 64))                            # residual's dtype
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w[:32])                                           # weight's length
    with pytest.raises(TypeError):
        ops.fp8_rmsnorm_quant_1x128(x, w.half())
    with pytest.raises(TypeError):
        ops.fp4_quant_1x32(x.half())
    with pytest.raises(ValueError):
        ops.fp4_rmsnorm_quant_1x32(x, w, out=ops.rmsnorm_quant_buffers(x, residual=True, bits=4))   # h without residual
    with pytest.raises(ValueError):
        ops.fp4_quant_1x32(x, scale=ops.fp4_scale_tiles(4, 256, "cpu"))                  # tiles of another matrix
    with pytest.raises(ValueError):
        ops.fp4_quant_1x32(x.t())                                                        # not row-major
    q, s = torch.zeros(4, 32, dtype=torch.uint8), ops.fp4_scale_tiles(4, 64, "cpu")
    with pytest.raises(ValueError):
        ops.fp4_scaled_gemm(q, torch.zeros(8, 16, dtype=torch.uint8), s, s)              # another K
    with pytest.raises(TypeError):
        ops.fp4_scaled_gemm(q.float(), q, s, s)
    with pytest.raises(ValueError):
        ops.fp8bs_rmsnorm_backward(x, x.float(), w, torch.ones(4))                       # dy's dtype


def test_binding_refuses_other_arguments():
    """What is no tensor, no number, on no GPU, or laid out otherwise raises; nothing is called."""
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    q, s, _, rstd, _ = out = ops.rmsnorm_quant_buffers(x)
    with pytest.raises(ValueError, match="CUDA"):
        ops.fp8_rmsnorm_quant_1x128(x, w, out=out)
    with pytest.raises(TypeError):
        ops.fp8_rmsnorm_quant_1x128(x, [1.0] * 256, out=out)
    with pytest.raises(TypeError):
        ops.fp8_rmsnorm_quant_1x128(x, w, eps="small", out=out)
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w, out=(q, s.contiguous(), None, rstd, None))       # a row-major grid
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w, out=(q, s, None, rstd.double(), None))
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(x, w, out=(q[:, :128], s, None, rstd, None))
    with pytest.raises(ValueError):
        ops.fp8_rmsnorm_quant_1x128(torch.zeros(256, dtype=torch.bfloat16), w)              # no matrix
    with pytest.raises(ValueError):
        ops.rmsnorm_quant_buffers(x, bits=6)
    c, t = torch.zeros(4, 128, dtype=torch.uint8), ops.fp4_scale_tiles(4, 256, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ops.fp4_scaled_gemm(c, c, t, t)
    with pytest.raises(ValueError):
        ops.fp4_scaled_gemm(c, c, t, t, out=torch.zeros(4, 5, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        ops.fp4_scaled_gemm(c, c, t, t, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.fp4_scaled_gemm(c, c, t, t[..., :2])
    with pytest.raises(TypeError):
        ops.fp4_dequant_1x32(c, t, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        ops.fp8bs_rmsnorm_backward(x, x, w, rstd, out=(x.clone(), torch.zeros(128)))
    with pytest.raises(TypeError):
        ops._load_native().norm(8, 0, x)                                                    # too few arguments
