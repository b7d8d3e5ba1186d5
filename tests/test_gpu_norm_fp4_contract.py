"""What include/fp8bs.h states about the norm's and the 4-bit calls at the edges of
their contract: values out of range, workspaces that do not fit, outputs over
inputs.  Every comparison is bit for bit."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from fp8_block_scaled_11_b200 import build, ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    ops.lib()


# ------------------------------------------------------------------ a value of y past fp32
@pytest.mark.parametrize("rows,cols", [(3, 512), (300, 8192), (310, 2080), (2, 16640)])
@pytest.mark.parametrize("how", ["8", "8pow2", "4"])
def test_norm_value_past_fp32(rows, cols, how):
    """A weight near fp32's limit: where y overflows, its group and no other is NaN once dequantized; rstd is as ever."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, cols, generator=g)
    x[:, 200] = 0.0
    x[1, 200] = 3.0                        # rstd is near 1: y = 3 x 3e38 there, 0 in every other row
    x = x.bfloat16().cuda()
    w = (1.0 + 0.2 * torch.randn(cols, generator=g)).cuda()
    big = w.clone()
    big[200] = 3e38

    def call(weight):
        if how == "4":
            return ops.fp4_rmsnorm_quant_1x32(x, weight, eps=EPS, want_y=True)
        return ops.fp8_rmsnorm_quant_1x128(x, weight, eps=EPS, want_y=True,
                                           rule=ops.SCALE_RULE_POW2 if how == "8pow2" else ops.SCALE_RULE_FP32)

    def values(q, s):
        if how == "4":
            return ops.fp4_dequant_1x32(q, s, out_dtype=torch.float32)
        return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)[:, :cols]
    q, s, _, rstd, y = call(w)
    qb, sb, _, rb, yb = call(big)
    assert torch.equal(rstd, rb) and bool(torch.isfinite(rb).all())
    assert bool(torch.isinf(yb[1, 200])) and int((y != yb).sum()) == 1
    width = 32 if how == "4" else 128
    hit = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    hit[1, 200 // width * width:200 // width * width + width] = True
    v, vb = values(q, s), values(qb, sb)
    assert torch.equal(torch.isnan(vb), hit)
    assert torch.equal(v[~hit], vb[~hit])
    if how == "4":
        e = sb.cpu().numpy().reshape(-1)[ref.tile_index(rows, cols // 32)]
        assert e[1, 200 // 32] == 255 and np.sum(e == 255) == 1
    else:
        assert bool(torch.isinf(sb[1, 1])) and int(torch.isinf(sb).sum()) == 1
