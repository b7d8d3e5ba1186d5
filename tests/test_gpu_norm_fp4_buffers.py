"""Workspaces that do not fit, and gradients written over their inputs.  A call that
is refused launches nothing; what it would have written stays.  Every comparison is
bit for bit."""
import pytest
import torch

from fp8_block_scaled_11_b200 import build, ops

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ALIGNMENT, WORKSPACE = 3, 4
# one cluster for all rows (a whole block of rows, and a remainder), rows over the ring (one CTA's threads, and
# over 256 of them), rows too wide for it
SHAPES = [(64, 512), (100, 64), (253, 128), (700, 1040), (300, 8192), (5, 16400)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    ops.lib()


def gradients(rows, cols, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    dy, h, dh = (torch.randn(rows, cols, generator=g).to(DT[dtype]).cuda() for _ in range(3))
    w = (1.0 + 0.2 * torch.randn(cols, generator=g)).to(DT[dtype]).cuda()
    return dy, h, w, (0.5 + torch.rand(rows, generator=g)).cuda(), dh


def refused(status, call):
    with pytest.raises(ops.Fp8bsError) as e:
        call()
    assert e.value.status == status


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_workspace_that_does_not_fit(rows, cols):
    dy, h, w, rstd, dh = gradients(rows, cols, "bf16")
    n = ops.rmsnorm_backward_workspace(h).numel()
    dx, dw = torch.full_like(h, 7.0), torch.full((cols,), 7.0, device="cuda")
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    refused(WORKSPACE, lambda: ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh, (dx, dw), buf[:n - 1]))
    refused(WORKSPACE, lambda: ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh, (dx, dw), buf[:0]))
    refused(ALIGNMENT, lambda: ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh, (dx, dw), buf[8:]))
    # none at all: the C entry point's answer (ops allocates one)
    assert ops._load_native().norm_backward(dy, h, w, rstd, dh, dx, dw, None) == WORKSPACE
    torch.cuda.synchronize()
    assert bool((dx == 7.0).all()) and bool((dw == 7.0).all()) and bool((buf == 0xA5).all())
    # the size that it asks for is enough
    want = ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh)
    got = ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh, (dx, dw), buf[:n])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buf[n:] == 0xA5).all())


@pytest.mark.parametrize("M,N,K", [(24, 100, 65568), (300, 100, 70016)])
def test_product_workspace_that_does_not_fit(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(5)
    a, b = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, device="cuda", generator=g) for n in (M, N))
    sa, sb = (torch.full_like(ops.fp4_scale_tiles(n, K, "cuda"), 127) for n in (M, N))
    n = ops.fp4_scaled_gemm_workspace(M, N, K, "cuda").numel()
    out = torch.full((M, N), 7.0, device="cuda")
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    refused(WORKSPACE, lambda: ops.fp4_scaled_gemm(a, b, sa, sb, out=out, workspace=buf[:n - 1]))
    refused(ALIGNMENT, lambda: ops.fp4_scaled_gemm(a, b, sa, sb, out=out, workspace=buf[8:]))
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and bool((buf == 0xA5).all())
    # sums of multiples of 1/4 below 2^22: exact, with K split over the workspace and without
    assert 36 * K < 2 ** 22
    ops.fp4_scaled_gemm(a, b, sa, sb, out=out, workspace=buf[:n])
    assert bool((buf[n:] == 0xA5).all()) and bool((buf[:n] != 0xA5).any())
    assert torch.equal(out, ops.fp4_scaled_gemm(a, b, sa, sb, out_dtype=torch.float32, split_k=False))


@pytest.mark.parametrize("over", ["dy", "h", "dh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gradient_over_its_inputs(rows, cols, dtype, over):
    dy, h, w, rstd, dh = gradients(rows, cols, dtype, rows)
    want = ops.fp8bs_rmsnorm_backward(dy, h, w, rstd, dh)
    buf = torch.full((rows, cols + 8), 7.0, dtype=DT[dtype], device="cuda")
    dx = buf[:, :cols]
    given = {"dy": dy, "h": h, "dh": dh}
    dx.copy_(given[over])
    given[over] = dx
    got = ops.fp8bs_rmsnorm_backward(given["dy"], given["h"], w, rstd, given["dh"], (dx, torch.empty(cols, device="cuda")))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buf[:, cols:] == 7.0).all())
