"""Microscaled 4-bit quantization, its inverse and the 4-bit product against
plain 64-bit forms (tests/mx4_reference.py).

Tolerances.  Quantization and dequantization have one exact answer: compared bit
for bit.  The product: products of codes and power-of-two factors are exact; the
fp32 accumulator takes ceil(K/64) additions (and as many splits' partial sums),
each losing at most 2^-22 of the largest partial sum, which S = sum |a||b|
bounds (the tensor cores may cut off below the last of 24 bits, hence a whole
step of 2^-23 and as much again for aligning the 64 products of a step).  bf16
output: half a step more, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from fp8_block_scaled_11_b200 import build, ops

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    ops.lib()


def no_device_error():
    st = ops.fp8bs_check_device_error()
    assert st == 0, ops.fp8bs_status_string(st)


def values(rows, cols, seed, dtype):
    """Normal values whose size varies by group, with borders, zeros, signed zeros, tiny and huge groups among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    flat = x.view(-1)
    flat[::7] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 3.0, -0.0, -2.5])[
        torch.randint(0, 11, (flat[::7].numel(),), generator=g)]
    x[0, :min(32, cols)] = 0.0
    if rows > 2:
        x[1] = -0.0
        x[2] = x[2] * 1e-30
    if rows > 4:
        x[3] = x[3] * (1e37 / x[3].abs().max())
        x[4, ::32] = 1.5 * 2.0 ** 20
    return x.to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 8192), (3, 64), (33, 160), (127, 128), (128, 96), (129, 1056),
                                       (300, 2080), (513, 256)])
def test_quant_rows(rows, cols, dtype):
    x = values(rows, cols, rows + 3 * cols, DT[dtype])
    q, s = ops.fp4_quant_1x32(x.cuda())
    code, e = ref.quant(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), ref.pack(code))
    got = s.cpu().numpy().reshape(-1)
    pad = np.full((rows, (cols + 127) // 128 * 4), 127, dtype=np.uint8)      # groups past the last: a scale of one
    pad[:, :cols // 32] = e
    assert np.array_equal(got[ref.tile_index(rows, pad.shape[1])], pad)
    v = ops.fp4_dequant_1x32(q, s, out_dtype=torch.float32)
    assert np.array_equal(v.cpu().double().numpy(), ref.value(code, e))
    v = ops.fp4_dequant_1x32(q, s)          # bf16 holds every value here but those past its range
    assert np.array_equal(v.cpu().double().numpy(), torch.from_numpy(ref.value(code, e)).bfloat16().double().numpy())
    no_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(32, 16), (32, 1040), (64, 128), (160, 48), (128, 256), (2080, 144)])
def test_quant_transposed(rows, cols, dtype):
    x = values(rows, cols, 5 * rows + cols, DT[dtype])
    q, s = ops.fp4_quant_1x32(x.cuda(), transpose_out=True)
    code, e = ref.quant(x.double().t().contiguous().numpy())
    assert np.array_equal(q.cpu().numpy(), ref.pack(code))
    pad = np.full((cols, (rows + 127) // 128 * 4), 127, dtype=np.uint8)
    pad[:, :rows // 32] = e
    assert np.array_equal(s.cpu().numpy().reshape(-1)[ref.tile_index(cols, pad.shape[1])], pad)


def test_quant_every_border():
    """Each code's borders and their neighbours, both signs, with the group's scale held by a 6."""
    mids = (ref.CODES[1:] + ref.CODES[:-1]) / 2
    t = np.concatenate([ref.CODES, mids, np.nextafter(mids.astype(np.float32), np.float32(0)),
                        np.nextafter(mids.astype(np.float32), np.float32(9))]).astype(np.float32)
    t = np.concatenate([t, -t])
    x = np.zeros((len(t), 32), dtype=np.float32)
    x[:, 0], x[:, 1] = 6.0, t
    q, s = ops.fp4_quant_1x32(torch.from_numpy(x).cuda())
    code, e = ref.quant(x.astype(np.float64))
    assert np.array_equal(ref.unpack(q.cpu().numpy()), code) and np.all(e == 127)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(256, 256), (160, 96)])
def test_quant_nan_and_infinity(rows, cols, dtype, transpose):
    """A group with a NaN or an infinity has the NaN scale and NaN values; every other group is as without them."""
    x = values(rows, cols, rows, DT[dtype])
    bad = x.clone()
    at = [(0, 0, float("nan")), (5, 95, float("inf")), (37, 40, -float("inf")), (rows - 1, cols - 1, -float("nan")),
          (130, 64, float("inf")), (130, 65, float("nan"))]
    hit = torch.zeros(rows, cols, dtype=torch.bool)
    for i, j, v in at:
        bad[i, j] = v
        if transpose:
            hit[i // 32 * 32:i // 32 * 32 + 32, j] = True
        else:
            hit[i, j // 32 * 32:j // 32 * 32 + 32] = True
    q, s = ops.fp4_quant_1x32(x.cuda(), transpose_out=transpose)
    qb, sb = ops.fp4_quant_1x32(bad.cuda(), transpose_out=transpose)
    v, vb = (ops.fp4_dequant_1x32(*t, out_dtype=torch.float32).cpu() for t in ((q, s), (qb, sb)))
    hit = hit.t() if transpose else hit
    assert torch.equal(torch.isnan(vb), hit) and torch.equal(v[~hit], vb[~hit])
    R, C = hit.shape
    e = sb.cpu().numpy().reshape(-1)[ref.tile_index(R, C // 32)]
    assert np.array_equal(e == 255, hit.reshape(R, C // 32, 32).any(2).numpy())


def test_quant_strides_and_guards():
    """Views with pitches: nothing outside the matrix is written, and scale bytes past the last row stay."""
    rows, cols = 130, 96
    big = values(rows, 160, 7, torch.bfloat16).cuda()
    x = big[:, 32:32 + cols]
    qbuf = torch.full((rows + 1, 64), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((2, 1, 32, 4, 4), 0xA5, dtype=torch.uint8, device="cuda")
    ops.fp4_quant_1x32(x, q=qbuf[:rows, :cols // 2], scale=s)
    code, e = ref.quant(x.cpu().double().numpy())
    got = qbuf.cpu().numpy()
    assert np.array_equal(got[:rows, :cols // 2], ref.pack(code))
    assert np.all(got[:rows, cols // 2:] == 0xA5) and np.all(got[rows:] == 0xA5)
    at = np.zeros(1024, dtype=bool)
    at[ref.tile_index(rows, 4)] = True
    assert np.all(s.cpu().numpy().reshape(-1)[~at] == 0xA5)
    out = torch.full((rows, 104), -7.0, dtype=torch.float32, device="cuda")
    ops.fp4_dequant_1x32(qbuf[:rows, :cols // 2], s, out=out[:, :cols])
    assert np.array_equal(out[:, :cols].cpu().double().numpy(), ref.value(code, e))
    assert bool((out[:, cols:] == -7.0).all())


# ------------------------------------------------------------------ product
def operand(rows, k, seed, spread=6, stale=None):
    """Random codes, scales over 2^+-spread, and their tiles; bytes of rows past the last are `stale` (NaN: 255)."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, size=(rows, k), dtype=np.uint8)
    e = (127 + rng.integers(-spread, spread + 1, size=(rows, k // 32))).astype(np.uint8)
    pad = np.full((rows, (k + 127) // 128 * 4), 127, dtype=np.uint8)
    pad[:, :k // 32] = e
    t = ref.tiles(pad, fill=255 if stale is None else stale)
    shape = ((rows + 127) // 128, (k + 127) // 128, 32, 4, 4)
    return (torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(t.reshape(shape)).cuda(), ref.value(code, e))


def check(got, a, b, out_dtype, k, splits=64):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2.0 ** -22 * (k / 64 + splits) * size
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{(err > tol).sum()} of {err.size} outside, worst {np.max(err / np.maximum(tol, 1e-300)):.2f} x"


SHAPES = [(1, 1, 32), (1, 5120, 8192), (7, 130, 96), (16, 128, 256), (17, 1000, 288), (33, 257, 4128), (64, 512, 512),
          (65, 300, 160), (128, 128, 2048), (129, 384, 1056), (200, 640, 224), (256, 4096, 1024), (300, 1000, 2080),
          (777, 1000, 2080), (1024, 19000, 64), (129, 19000, 96), (2300, 2304, 288),
          (5000, 1100, 544), (2305, 2050, 4128), (70, 19000, 160), (1, 100, 1056), (5, 100, 2080), (20, 130, 2080),
          (40, 100, 2080), (65, 100, 4128), (500, 520, 8224), (4000, 2050, 96), (20, 100, 4128), (300, 4100, 8192),
          (1500, 130, 16416)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, dtype):
    a, sa, av = operand(M, K, M + N + K)
    b, sb, bv = operand(N, K, M + N + K + 1)
    d = ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=DT[dtype])
    no_device_error()
    check(d, av, bv, DT[dtype], K)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact(M, N, K):
    """Scales of one: every sum is a multiple of 1/4 below 2^22, so fp32 holds it exactly, whatever the order."""
    a, sa, av = operand(M, K, 2 * M + N + K, spread=0)
    b, sb, bv = operand(N, K, 3 * M + N + K, spread=0)
    assert 36 * K < 2 ** 22
    d = ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32)
    no_device_error()
    assert np.array_equal(d.double().cpu().numpy(), av @ bv.T)
    d2 = ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32, split_k=False)
    no_device_error()
    assert torch.equal(d, d2)


@pytest.mark.parametrize("M,N,K", [(5000, 4200, 8192), (16640, 1300, 4128), (300, 40000, 1600), (65, 5000, 3104),
                                   (65, 5000, 12320), (529, 2050, 8224), (500, 520, 32800), (24, 100, 65568),
                                   (2048, 4096, 1056), (2600, 4100, 32), (1600, 5200, 4160)])
def test_product_exact_large(M, N, K):
    """Many tiles per CTA, many steps per tile, K split over clusters of two, four and eight CTAs at every tile width
    and through the workspace; the reference in 64 bits on the GPU: exact as above."""
    assert 36 * K < 2 ** 22
    a, sa, av = operand(M, K, 51, spread=0)
    b, sb, bv = operand(N, K, 52, spread=0)
    want = (torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t())
    assert torch.equal(ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32).double(), want)
    assert torch.equal(ops.fp4_scaled_gemm(a, b, sa, sb), want.float().bfloat16())
    no_device_error()


@pytest.mark.parametrize("M,N,K,ldd", [(5, 70, 96, 75), (130, 257, 320, 301), (300, 130, 256, 131), (700, 515, 320, 517),
                                       (260, 20000, 96, 20004)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_product_strides_and_guards(M, N, K, ldd, dtype):
    """Pitched operands and an odd output pitch; nothing outside D is written."""
    a, sa, av = operand(M, K, 11)
    b, sb, bv = operand(N, K, 12)
    pitch = (K // 2 + 15) // 16 * 16 + 32
    ap = torch.full((M, pitch), 0xFF, dtype=torch.uint8, device="cuda")
    bp = torch.full((N, pitch), 0xFF, dtype=torch.uint8, device="cuda")
    ap[:, :K // 2] = a
    bp[:, :K // 2] = b
    buf = torch.full((M + 1, ldd), -7.0, dtype=DT[dtype], device="cuda")
    ops.fp4_scaled_gemm(ap[:, :K // 2], bp[:, :K // 2], sa, sb, out=buf[:M, :N])
    no_device_error()
    check(buf[:M, :N], av, bv, DT[dtype], K)
    assert bool((buf[:M, N:] == -7.0).all()) and bool((buf[M:] == -7.0).all())


def test_one_row_with_any_stride():
    """One token taken out of a larger tensor, and a row whose stride is meaningless."""
    N, K = 300, 512
    big, sbig, bv = operand(9, K, 61)
    b, sb, bw = operand(N, K, 62)
    q = torch.as_strided(big, (1, K // 2), (1, 1), 4 * (K // 2))       # row 4
    x = ops.fp4_dequant_1x32(big, sbig)[4:5]
    qa, sa = ops.fp4_quant_1x32(x)                                      # the same values again
    va = ops.fp4_dequant_1x32(qa, sa, out_dtype=torch.float32)
    assert torch.equal(va, x.float())
    d = ops.fp4_scaled_gemm(torch.as_strided(qa, (1, K // 2), (3, 1)), b, sa, sb, out_dtype=torch.float32)
    check(d, bv[4:5], bw, torch.float32, K)
    s4 = ops.fp4_scale_tiles(1, K, "cuda")
    s4[0, :, 0, 0] = sbig[0, :, 4, 0]
    d = ops.fp4_scaled_gemm(q, b, s4, sb, out_dtype=torch.float32)
    no_device_error()
    check(d, bv[4:5], bw, torch.float32, K)


def test_product_nan_scale_stays_in_its_row():
    """A NaN scale (255) in one row of A makes that row of D NaN and no other."""
    M, N, K = 40, 200, 512
    a, sa, av = operand(M, K, 21)
    b, sb, bv = operand(N, K, 22)
    sa.view(-1)[int(ref.tile_index(M, 16)[9, 5])] = 255
    d = ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32)
    no_device_error()
    assert bool(torch.isnan(d[9]).all())
    keep = [i for i in range(M) if i != 9]
    check(d[keep], av[keep], bv, torch.float32, K)


@pytest.mark.parametrize("M,N,K", [(24, 256, 65536 + 32), (1, 130, 131072), (100, 100, 65536), (300, 100, 70016)])
def test_product_long_k(M, N, K):
    a, sa, av = operand(M, K, 31, spread=2)
    b, sb, bv = operand(N, K, 32, spread=2)
    d = ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32)
    no_device_error()
    check(d, av, bv, torch.float32, K)


def test_product_deterministic_and_captured():
    """Twice the same bits; the same from a replayed graph, on another stream."""
    M, N, K = 8, 1024, 8192
    a, sa, _ = operand(M, K, 41)
    b, sb, _ = operand(N, K, 42)
    ws = ops.fp4_scaled_gemm_workspace(M, N, K, "cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    first = ops.fp4_scaled_gemm(a, b, sa, sb, workspace=ws).clone()
    assert torch.equal(first, ops.fp4_scaled_gemm(a, b, sa, sb, workspace=ws))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.fp4_scaled_gemm(a, b, sa, sb, out=out, workspace=ws)
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.replay()
        g.replay()
    side.synchronize()
    assert torch.equal(first, out)
    no_device_error()


def test_past_32_bit_offsets():
    """More than 2^31 elements: the last rows equal the same rows on their own; the last columns too."""
    rows, cols, tail = 131200, 16384, 256
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(2))
    q, s = ops.fp4_quant_1x32(x)
    q1, s1 = ops.fp4_quant_1x32(x[-tail:])
    assert torch.equal(q[-tail:], q1) and torch.equal(s[-tail // 128:], s1)
    v = ops.fp4_dequant_1x32(q, s)
    assert torch.equal(v[-tail:], ops.fp4_dequant_1x32(q1, s1))
    del v
    qt, st = ops.fp4_quant_1x32(x, transpose_out=True)
    qt1, st1 = ops.fp4_quant_1x32(x[:, -128:], transpose_out=True)
    assert torch.equal(qt[-128:], qt1) and torch.equal(st[-1:], st1)
    # D of 70016 x 32000 bf16; codes of small integers and scales of one: every sum is exact in any order
    M, N, K = 70016, 32000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = (torch.randint(0, 256, (n, K // 2), device="cuda", dtype=torch.uint8, generator=g) for n in (M, N))
    sa, sb = (torch.full_like(ops.fp4_scale_tiles(n, K, "cuda"), 127) for n in (M, N))
    d = ops.fp4_scaled_gemm(a, b, sa, sb)
    d1 = ops.fp4_scaled_gemm(a[-tail:], b, sa[-tail // 128:].contiguous(), sb)
    no_device_error()
    assert torch.equal(d[-tail:], d1)
