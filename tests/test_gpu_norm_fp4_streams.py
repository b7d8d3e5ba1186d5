"""Calls on two streams that fork and join by events: a programmatic launch whose
stream has just waited for another one's kernel, a copy or a memset.  The same bits
as one after the other, eagerly and from a replayed graph."""
import pytest
import torch

from fp8_block_scaled_11_b200 import build, inputs, ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 24, 300, 2300])
def test_fork_and_join(M):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    K = 1024
    x0, r0 = (inputs.random_matrix(M, K, seed=s).cuda() for s in (61, 62))
    w0 = inputs.random_matrix(K, K, seed=63, scale=K ** -0.5).cuda()
    g0 = torch.linspace(0.5, 1.5, K, device="cuda").bfloat16()
    x, r, g, w = (torch.empty_like(t) for t in (x0, r0, g0, w0))
    wq, ws = ops.fp4_quant_1x32(w0)
    rq, rs = ops.fp4_quant_1x32(r0)
    out = ops.rmsnorm_quant_buffers(x0, residual=True, bits=4)
    dx, dw, d = torch.empty_like(x0), torch.empty(K, device="cuda"), torch.empty((M, K), dtype=x0.dtype, device="cuda")
    bwd = ops.rmsnorm_backward_workspace(x0)
    side = torch.cuda.Stream()

    def steps(fork):
        """fork: what runs beside the main stream runs on `side`; else all of it in one row, waited for."""
        main = torch.cuda.current_stream()
        x.copy_(x0)
        r.copy_(r0)
        g.copy_(g0)
        w.copy_(w0)
        for i in range(40):
            beside = side if fork else main
            beside.wait_stream(main)
            with torch.cuda.stream(beside):
                # the weight and its codes, the residual and the norm's weight, while the main stream does the rest
                w.mul_(-1.0)
                ops.fp4_quant_1x32(w, q=wq, scale=ws)
                ops.fp4_quant_1x32(r, q=rq, scale=rs)
                ops.fp4_dequant_1x32(rq, rs, out=r)
                if i % 3 == 2:
                    g.copy_(g0)             # a copy, not a kernel, in front of the join
            if not fork:
                torch.cuda.synchronize()
            d.zero_()
            main.wait_stream(beside)
            _, _, h, rstd, _ = ops.fp4_rmsnorm_quant_1x32(x, g, residual=r, out=out)
            ops.fp4_scaled_gemm(out[0], wq, out[1], ws, out=d)
            ops.fp8bs_rmsnorm_backward(d, h, g, rstd, dh=r, out=(dx, dw), workspace=bwd)
            if not fork:
                torch.cuda.synchronize()
            x.copy_(dx)
            g.add_(dw.to(g.dtype), alpha=1e-3)
        return [t.clone() for t in (x, r, g, d, out[0], out[3], dw)]

    want = steps(False)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    got = steps(True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = steps(True)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, want))
    assert ops.fp8bs_check_device_error() == 0
