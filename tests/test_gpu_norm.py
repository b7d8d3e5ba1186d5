"""The RMS norm with a quantized result and its backward pass against plain
64-bit forms (tests/mx4_reference.py).

Tolerances (u = 2^-24, a rounding of fp32).  h: the sum of two values in x's
type, one rounding of an fp32 sum: equal.  Sum of squares: all terms positive; a
thread adds at most 32 + cols/512 of them one after another, then at most 16
levels: relative error below (cols/512 + 48) u; rstd takes half of it and three
roundings; y three more.  A scale takes y's error, a division and a reciprocal.
An 8-bit value is within half a step (2^-4 of it, or 2^-10 where it is
subnormal), a 4-bit one within a quarter, a half or one (half the distance
between codes), of y times the scale that was stored.
Backward: dx is a handful of roundings of each of its three terms, with the
mean's error (cols u of mean |g n| at most); dweight adds rows terms: rows u of
sum |dy n| at most.  Outputs in bf16: 2^-8 of the value more."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from fp8_block_scaled_11_b200 import build, ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    ops.lib()


def make(rows, cols, dtype, seed, wdtype=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(DT[dtype])
    r = torch.randn(rows, cols, generator=g).to(DT[dtype])
    w = (1.0 + 0.2 * torch.randn(cols, generator=g)).to(DT[wdtype or dtype])
    x[0, ::5] *= 100.0
    return x, r, w


def rel_rstd(cols):
    return ((cols / 512 + 48) / 2 + 3) * U


def check_forward(x, r, w, got, bits, pow2=False):
    rows, cols = x.shape
    q, s, h, rstd, y = got
    h0, rstd0, y0 = ref.norm(x, r, w, EPS)
    assert torch.equal(h.cpu(), h0)
    tol = rel_rstd(cols)
    assert bool(((rstd.cpu().double() - rstd0).abs() <= tol * rstd0).all())
    tol += 3 * U
    if y is not None:
        half = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
        assert bool(((y.cpu().double() - y0).abs() <= (tol + half) * y0.abs()).all())
    y0 = y0.numpy()
    if bits == 8:
        pad = np.zeros((rows, (cols + 127) // 128 * 128))
        pad[:, :cols] = np.abs(y0)
        amax = np.maximum(pad.reshape(rows, -1, 128).max(2), 1e-12)
        scale = s.cpu().double().numpy()
        if pow2:
            m, _ = np.frexp(scale)
            assert np.all(m == 0.5)
            assert np.all(scale >= amax / 448 * (1 - tol - 2 * U)) and np.all(scale < 2 * amax / 448 * (1 + tol + 2 * U))
        else:
            assert np.all(np.abs(scale - amax / 448) <= (tol + 2 * U) * amax / 448)
        t = y0 / np.repeat(scale, 128, 1)[:, :cols]
        v = q.view(torch.float8_e4m3fn).cpu().double().numpy()
        assert np.all(np.abs(v - t) <= np.maximum(np.abs(t) * 2.0 ** -4, 2.0 ** -10) + np.abs(t) * (tol + 4 * U))
    else:
        e = s.cpu().numpy().reshape(-1)[ref.tile_index(rows, (cols + 127) // 128 * 4)]
        assert np.all(e[:, cols // 32:] == 127)
        scale = np.ldexp(1.0, e[:, :cols // 32].astype(np.int64) - 127)
        amax = np.maximum(np.abs(y0).reshape(rows, -1, 32).max(2), 1e-12)
        assert np.all(amax <= 6 * scale * (1 + tol)) and np.all(amax > 3 * scale * (1 - tol))
        t = np.abs(y0 / np.repeat(scale, 32, 1))
        code = ref.unpack(q.cpu().numpy())
        v = ref.CODES[code & 7]
        half = np.where(t <= 2 * (1 + tol), 0.25, np.where(t <= 4 * (1 + tol), 0.5, 1.0))
        assert np.all(np.abs(v - t) <= half + t * tol)
        assert np.array_equal(code >> 3, np.signbit(y0).astype(np.uint8))


SHAPES = [(1, 32), (1, 5120), (1, 8192), (2, 160), (3, 16384), (31, 96), (300, 2080), (299, 8192), (777, 2048),
          (350, 4128), (1500, 128), (1031, 32), (4, 16416), (301, 20000 // 32 * 32)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype, bits):
    x, r, w = make(rows, cols, dtype, rows + cols)
    fn = ops.fp8_rmsnorm_quant_1x128 if bits == 8 else ops.fp4_rmsnorm_quant_1x32
    with_r = fn(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    check_forward(x, r, w, with_r, bits)
    without = fn(x.cuda(), w.cuda(), eps=EPS, want_y=True)
    check_forward(x, None, w, without, bits)


@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 144), (400, 1040), (3, 16400)])
def test_forward_ragged_group_and_pow2(rows, cols):
    x, r, w = make(rows, cols, "bf16", rows * cols, wdtype="fp32")
    got = ops.fp8_rmsnorm_quant_1x128(x.cuda(), w.cuda(), r.cuda(), eps=EPS, rule=ops.SCALE_RULE_POW2, want_y=True)
    check_forward(x, r, w, got, 8, pow2=True)


def test_forward_zero_rows():
    """A row of zeros: h / sqrt(eps) = 0, codes of zero, the scale of the smallest group maximum."""
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    x[1] = 1.0
    w = torch.ones(256, dtype=torch.bfloat16)
    q, s, _, rstd, _ = ops.fp8_rmsnorm_quant_1x128(x.cuda(), w.cuda(), eps=EPS)
    assert bool((q[0] == 0).all()) and bool((q[2] == 0).all()) and bool((q[1] != 0).all())
    assert abs(float(rstd[0]) - 1e3) < 1e-2 and bool(torch.isfinite(s).all())
    q, s, _, _, _ = ops.fp4_rmsnorm_quant_1x32(x.cuda(), w.cuda(), eps=EPS)
    assert bool((q[0] == 0).all()) and bool((q[1] != 0).all())


@pytest.mark.parametrize("rows,cols", [(3, 512), (300, 8192), (310, 2080), (2, 16640)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e25])
def test_forward_row_out_of_range(rows, cols, value):
    """A NaN, an infinity or a sum of squares past fp32 makes its row NaN in either format, and no other row."""
    x, r, w = make(rows, cols, "bf16", 11)
    bad = x.clone()
    bad[1, 37] = value
    keep = [i for i in range(rows) if i != 1]
    for bits, fn in ((8, ops.fp8_rmsnorm_quant_1x128), (4, ops.fp4_rmsnorm_quant_1x32)):
        q, s, _, rstd, _ = fn(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
        qb, sb, _, rb, _ = fn(bad.cuda(), w.cuda(), r.cuda(), eps=EPS)
        assert torch.equal(q[keep], qb[keep]) and torch.equal(rstd[keep], rb[keep]) and bool(torch.isnan(rb[1]))
        if bits == 8:
            assert bool(torch.isnan(qb.view(torch.float8_e4m3fn).float()[1]).all())
        else:
            assert bool(torch.isnan(ops.fp4_dequant_1x32(qb, sb)[1]).all())
            assert torch.equal(ops.fp4_dequant_1x32(q, s)[keep], ops.fp4_dequant_1x32(qb, sb)[keep])


@pytest.mark.parametrize("rows,cols", [(3, 512), (300, 1024), (2, 16640)])
def test_forward_in_place_and_pitched(rows, cols):
    """h over the residual, and over x; pitched views; nothing else is written."""
    x, r, w = make(rows, cols, "bf16", 3)
    want = ops.fp8_rmsnorm_quant_1x128(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    for over in ("residual", "x"):
        xb = torch.full((rows, cols + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        rb = torch.full((rows, cols + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        xv, rv = xb[:, :cols], rb[:, :cols]
        xv.copy_(x)
        rv.copy_(r)
        q, s, _, rstd, _ = ops.rmsnorm_quant_buffers(x.cuda(), residual=True)
        qb = torch.full((rows, cols + 16), 9, dtype=torch.uint8, device="cuda")
        h = rv if over == "residual" else xv
        got = ops.fp8_rmsnorm_quant_1x128(xv, w.cuda(), rv, eps=EPS, out=(qb[:, :cols], s, h, rstd, None))
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)
        assert bool((qb[:, cols:] == 9).all()) and bool((xb[:, cols:] == 7).all()) and bool((rb[:, cols:] == 7).all())


# ------------------------------------------------------------------ backward
def check_backward(dy, h, w, rstd, dh, got):
    dx0, dw0 = ref.norm_backward(dy, h, w, rstd, dh)
    rows, cols = h.shape
    n = h.double() * rstd.double()[:, None]
    g = dy.double() * w.double()
    r = rstd.double()[:, None]
    size = r * (g.abs() + 2 * n.abs() * (g * n).abs().mean(1, keepdim=True))
    tol = 8 * U * size + r * n.abs() * cols * U * (g * n).abs().mean(1, keepdim=True)
    if dh is not None:
        tol = tol + U * (dh.double().abs() + size)
    half = 2.0 ** -8 if h.dtype == torch.bfloat16 else U
    dx, dw = got
    assert bool(((dx.cpu().double() - dx0).abs() <= tol + half * dx0.abs()).all())
    assert bool(((dw.cpu().double() - dw0).abs() <= (rows + 8) * U * (dy.double() * n).abs().sum(0)).all())


BACK = [(1, 16), (1, 8192), (2, 5120), (33, 144), (300, 1040), (1200, 256), (700, 8192), (2500, 2064), (5, 8208),
        (260, 16400), (3000, 128), (700, 96), (100, 64), (5, 1024), (60, 496), (250, 208)]


def back_inputs(rows, cols, dtype, seed, wdtype=None):
    h, dh, w = make(rows, cols, dtype, seed, wdtype)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    return dy, h, w, rstd, dh


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", BACK)
def test_backward(rows, cols, dtype, residual):
    dy, h, w, rstd, dh = back_inputs(rows, cols, dtype, rows + cols)
    dh = dh if residual else None
    got = ops.fp8bs_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=None if dh is None else dh.cuda())
    check_backward(dy, h, w, rstd, dh, got)
    again = ops.fp8bs_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=None if dh is None else dh.cuda())
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("rows,cols", [(3, 144), (300, 1040), (4, 16400)])
@pytest.mark.parametrize("power", [50, -50])
def test_backward_of_large_and_small_rows(rows, cols, power):
    """rstd is near 2^-50 or 2^50: its square is in fp32's range, its cube is not."""
    dy, h, w, _, _ = back_inputs(rows, cols, "fp32", rows + 7)
    h = torch.ldexp(h, torch.tensor(power))
    rstd = (1.0 / torch.sqrt(h.double().square().mean(1))).float()
    got = ops.fp8bs_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    check_backward(dy, h, w, rstd, None, got)


def test_backward_mixed_weight_pitched_in_place():
    rows, cols = 70, 528
    dy, h, w, rstd, dh = back_inputs(rows, cols, "bf16", 5, wdtype="fp32")
    buf = torch.full((rows, cols + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = buf[:, :cols]
    dx.copy_(dh)
    dw = torch.empty(cols, device="cuda")
    got = ops.fp8bs_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=dx, out=(dx, dw))
    check_backward(dy, h, w, rstd, dh, got)
    assert bool((buf[:, cols:] == 7.0).all())


def test_backward_against_differences():
    """Central differences, in 64 bits, of L = sum(y c) along random directions: dL/dx . v and dL/dw . u.  The
    differences' own error is of order step^2, far below the gradients' tolerance."""
    rows, cols = 6, 160
    c, h, w, _, _ = back_inputs(rows, cols, "fp32", 9)
    _, rstd, _, = ref.norm(h, None, w, EPS)
    dx, dw = ops.fp8bs_rmsnorm_backward(c.cuda(), h.cuda(), w.cuda(), rstd.float().cuda())
    rng = torch.Generator().manual_seed(1)

    def loss(x, wt):
        r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        return float((x * r * wt * c.double()).sum())
    for _ in range(4):
        v = torch.randn(rows, cols, generator=rng, dtype=torch.float64)
        u = torch.randn(cols, generator=rng, dtype=torch.float64)
        t = 1e-5
        num = (loss(h.double() + t * v, w.double()) - loss(h.double() - t * v, w.double())) / (2 * t)
        got = float((dx.cpu().double() * v).sum())
        assert abs(num - got) <= 1e-5 * float((dx.cpu().double() * v).abs().sum())
        num = (loss(h.double(), w.double() + t * u) - loss(h.double(), w.double() - t * u)) / (2 * t)
        got = float((dw.cpu().double() * u).sum())
        assert abs(num - got) <= 1e-5 * float((dw.cpu().double() * u).abs().sum())


# ------------------------------------------------------------------ together
def test_norm_then_product_8_and_4_bits():
    """A layer as a model runs it: norm, quantized result, product with the layer's weight.  The result is exactly
    the product of the quantized operands (each within its own tests' tolerance)."""
    rows, K, N = 150, 1024, 384
    x, r, w = make(rows, K, "bf16", 77)
    W = (torch.randn(N, K, generator=torch.Generator().manual_seed(78)) * K ** -0.5).bfloat16()
    q, s, h, rstd, _ = ops.fp8_rmsnorm_quant_1x128(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    wq, ws, _, _ = ops.fp8_quant_128x128(W.cuda())
    y = ops.fp8_scaled_gemm(q, wq, s, ws, ops.SCALE_BLOCK_1x128_128x128, out_dtype=torch.float32)
    a = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
    b = wq.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    assert float((y.double() - a @ b.t()).norm() / (a @ b.t()).norm()) < 1e-5
    _, _, y0 = ref.norm(x, r, w, EPS)
    full = y0 @ W.double().t()
    assert float((y.cpu().double() - full).norm() / full.norm()) < 0.13      # two factors, each value of either within 2^-4

    q4, s4, h4, _, _ = ops.fp4_rmsnorm_quant_1x32(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    assert torch.equal(h, h4)
    wq4, ws4 = ops.fp4_quant_1x32(W.cuda())
    y4 = ops.fp4_scaled_gemm(q4, wq4, s4, ws4, out_dtype=torch.float32)
    a = ops.fp4_dequant_1x32(q4, s4, out_dtype=torch.float32).double()
    b = ops.fp4_dequant_1x32(wq4, ws4, out_dtype=torch.float32).double()
    size = a.abs() @ b.abs().t()
    assert bool(((y4.double() - a @ b.t()).abs() <= 2.0 ** -22 * (K / 64 + 64) * size).all())
    # backward of the same layer: dgrad in 8 bits gives dy, the norm's backward takes it on
    dout = torch.randn(rows, N, generator=torch.Generator().manual_seed(79)).bfloat16().cuda()
    dq, ds = ops.fp8_quant_1x128(dout)
    dy = ops.fp8_scaled_gemm_ex(dq, wq, ops.MAJOR_MN, ds, ws, ops.SCALE_BLOCK_1x128_128x128)
    dx, dw = ops.fp8bs_rmsnorm_backward(dy, h, w.cuda(), rstd, dh=r.cuda())
    check_backward(dy.cpu(), h.cpu(), w, rstd.cpu(), r, (dx, dw))
    st = ops.fp8bs_check_device_error()
    assert st == 0, ops.fp8bs_status_string(st)


def test_past_32_bit_offsets():
    """More than 2^31 elements: the last rows equal the same rows on their own (each row's result is its own)."""
    rows, cols, tail = 131200, 16384, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16, generator=g)
    r = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16, generator=g)
    w = torch.randn(cols, device="cuda", generator=g).bfloat16()
    last = slice(rows - tail, rows)
    for fn in (ops.fp8_rmsnorm_quant_1x128, ops.fp4_rmsnorm_quant_1x32):
        q, s, h, rstd, _ = fn(x, w, r)
        q1, s1, h1, rstd1, _ = fn(x[last], w, r[last])
        assert torch.equal(q[last], q1) and torch.equal(h[last], h1) and torch.equal(rstd[last], rstd1)
        assert torch.equal(s[last] if s.dim() == 2 else s[-(tail // 128):], s1)
    dx, _ = ops.fp8bs_rmsnorm_backward(x, h, w, rstd, dh=r)
    dx1, _ = ops.fp8bs_rmsnorm_backward(x[last], h1, w, rstd1, dh=r[last])
    assert torch.equal(dx[last], dx1)


def test_captured_with_eager_alive():
    """Forward and backward captured into one graph while eager results live; replayed on new inputs, bit for bit."""
    rows, cols = 40, 1024
    x, r, w = (t.cuda() for t in make(rows, cols, "bf16", 5))
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    out = ops.rmsnorm_quant_buffers(x, residual=True)
    back = (torch.empty_like(x), torch.empty(cols, device="cuda"))
    ws = ops.rmsnorm_backward_workspace(x)

    def step():
        _, _, h, rstd, _ = ops.fp8_rmsnorm_quant_1x128(x, w, r, eps=EPS, out=out)
        ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh=r, out=back, workspace=ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*out[:4], *back)]
    step()
    for a, b in zip(got, (*out[:4], *back)):
        assert torch.equal(a, b)
