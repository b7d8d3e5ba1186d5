"""Python binding of libfp8bs (the C ABI in include/fp8bs.h).

Argument marshalling only: every function here checks the tensors' device,
allocates outputs with torch when they are not given, and calls the C entry
point of the same name with raw pointers and torch's current CUDA stream.  All
arithmetic happens in the CUDA library; if the library is missing or was not
built, the first call raises -- there is no fallback path.

Scale grids are column-major fp32, as the library writes and reads them.  In
torch they are returned as (rows, groups) views with strides (1, ld): element
[i, j] is the scale of row i, group j, stored at i + j*ld.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import torch

from . import build as _build

FP8BS_OK = 0
STATUS_NAMES = {
    0: "FP8BS_OK", 1: "FP8BS_ERR_INVALID_ARG", 2: "FP8BS_ERR_UNSUPPORTED", 3: "FP8BS_ERR_ALIGNMENT",
    4: "FP8BS_ERR_WORKSPACE", 5: "FP8BS_ERR_CUDA", 6: "FP8BS_ERR_TIMEOUT", 7: "FP8BS_ERR_NO_SM100",
    8: "FP8BS_ERR_SCALE",
}

BF16, F32 = 0, 1
SCALE_TENSOR, SCALE_ROWWISE, SCALE_BLOCK_1x128_128x128, SCALE_BLOCK_1x128_1x128 = 0, 1, 2, 3
# the block recipes with power-of-two scales on the block-scaled MMA
SCALE_BLOCK_1x128_128x128_POW2, SCALE_BLOCK_1x128_1x128_POW2 = 4, 5
BLOCK_MODES = (SCALE_BLOCK_1x128_128x128, SCALE_BLOCK_1x128_1x128,
               SCALE_BLOCK_1x128_128x128_POW2, SCALE_BLOCK_1x128_1x128_POW2)
SCALE_RULE_FP32, SCALE_RULE_POW2 = 0, 1
SCALE_COL_MAJOR = 0
MAJOR_K, MAJOR_MN = 0, 1

_lib = None


class Fp8bsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


def lib():
    """Load libfp8bs.so (built in-tree).  Raises if it is absent."""
    global _lib
    if _lib is None:
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise ImportError(f"libfp8bs.so not built ({path}); run fp8_block_scaled_11_b200/build.py")
        L = ctypes.CDLL(path)
        p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.fp8_quant_1x128.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, i32, p]
        L.fp8_quant_1x128_dual.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p]
        L.fp8_quant_128x128.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p]
        L.fp8_quant_1x128_ex.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, i32, i32, p]
        L.fp8_quant_1x128_dual_ex.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, p]
        L.fp8_quant_128x128_ex.argtypes = [p, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, p]
        L.fp8_quant_tensor_workspace_size.argtypes = [i64]
        L.fp8_quant_tensor_workspace_size.restype = sz
        L.fp8_quant_tensor.argtypes = [p, i32, i64, p, p, p, sz, p]
        L.fp8_quant_rowwise.argtypes = [p, i32, i64, i64, i64, p, i64, p, p]
        L.fp8_scaled_gemm_workspace_size.argtypes = [i64, i64, i64, i32]
        L.fp8_scaled_gemm_workspace_size.restype = sz
        L.fp8_scaled_gemm.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, i32, p, i64, i32, p, sz, p]
        L.fp8_scaled_gemm_ex.argtypes = [i64, i64, i64, p, i64, p, i64, i32, p, i64, p, i64, i32, i32, p, i64, i32,
                                         p, sz, p]
        L.fp8_scaled_gemm_grouped.argtypes = [i64, p, i64, i64, p, i64, p, i64, p, i64, p, i64, i64, i32, i32, p,
                                              i64, i32, p]
        L.fp8_scaled_gemm_quant.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, i32, p, i64,
                                            p, i64, p, i64, p]
        f32 = ctypes.c_float
        norm = [p, i64, p, i64, i32, i64, i64, p, i32, f32, p, i64, p, p, i64, p, i64, p]
        L.fp8_rmsnorm_quant_1x128.argtypes = norm + [i64, i32, p]
        L.fp4_rmsnorm_quant_1x32.argtypes = norm + [p]
        L.fp8bs_rmsnorm_backward_workspace_size.argtypes = [i64, i64]
        L.fp8bs_rmsnorm_backward.argtypes = [p, i64, p, i64, p, i64, i32, i64, i64, p, i32, p, p, i64, p, p, sz, p]
        L.fp4_scale_tiles_size.argtypes = [i64, i64]
        L.fp4_quant_1x32.argtypes = [p, i32, i64, i64, i64, p, i64, p, i32, p]
        L.fp4_dequant_1x32.argtypes = [p, i64, p, i64, i64, p, i32, i64, p]
        L.fp4_scaled_gemm_workspace_size.argtypes = [i64, i64, i64]
        L.fp4_scaled_gemm.argtypes = [i64, i64, i64, p, i64, p, i64, p, p, p, i64, i32, p, sz, p]
        for fn in ("fp8bs_rmsnorm_backward_workspace_size", "fp4_scale_tiles_size", "fp4_scaled_gemm_workspace_size"):
            getattr(L, fn).restype = sz
        L.fp8bs_status_string.argtypes = [i32]
        L.fp8bs_status_string.restype = ctypes.c_char_p
        L.fp8bs_check_device_error.argtypes = [p]
        L.fp8_quant_tensor_noalloc.argtypes = [p, i32, i64, p, p, p]
        for fn in ("fp8_quant_1x128", "fp8_quant_1x128_dual", "fp8_quant_128x128", "fp8_quant_1x128_ex",
                   "fp8_quant_1x128_dual_ex", "fp8_quant_128x128_ex", "fp8_quant_tensor",
                   "fp8_quant_rowwise", "fp8_scaled_gemm", "fp8_scaled_gemm_ex", "fp8_scaled_gemm_quant", "fp8_scaled_gemm_grouped",
                   "fp8bs_check_device_error", "fp8_quant_tensor_noalloc", "fp8_rmsnorm_quant_1x128",
                   "fp4_rmsnorm_quant_1x32", "fp8bs_rmsnorm_backward", "fp4_quant_1x32", "fp4_dequant_1x32",
                   "fp4_scaled_gemm"):
            getattr(L, fn).restype = i32
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != FP8BS_OK:
        raise Fp8bsError(fn, status)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported input dtype {t.dtype} (bf16 or fp32)")


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major tensor (unit column stride)")
    return t.stride(0)


def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def colmajor_grid(rows: int, groups: int, device) -> torch.Tensor:
    """Allocate a column-major fp32 scale grid (rows x groups), ld = rows rounded up to 4."""
    ld = _round_up(max(rows, 1), 4)
    return torch.empty((groups, ld), dtype=torch.float32, device=device)[:, :rows].t()


def _grid_ld(s: torch.Tensor, rows: int) -> int:
    if s.dim() != 2 or s.dtype != torch.float32:
        raise ValueError("scale grid must be a 2-D fp32 tensor")
    if s.shape[1] == 1:
        return s.stride(1) if s.stride(0) == 1 and s.stride(1) >= rows else _round_up(rows, 4)
    if s.stride(0) != 1:
        raise ValueError("scale grid must be column-major (stride (1, ld))")
    return s.stride(1)


# ---------------------------------------------------------------------------- quantization
def fp8_quant_1x128(x: torch.Tensor, transpose_out: bool = False, q: Optional[torch.Tensor] = None,
                    scale_inv: Optional[torch.Tensor] = None, rule: int = SCALE_RULE_FP32):
    """Returns (q uint8, scale_inv grid).  transpose_out=False: q is rows x cols,
    grid rows x ceil(cols/128).  transpose_out=True: groups run along rows and
    q is the quantized transpose (cols x rows), grid cols x ceil(rows/128).
    Preallocated outputs may be passed as q / scale_inv.  rule =
    SCALE_RULE_POW2 rounds every scale down to a power of two (fp8_quant_1x128_ex)."""
    rows, cols = x.shape
    xt = _dtype_code(x)
    out_rows, out_cols = (cols, rows) if transpose_out else (rows, cols)
    if q is None:
        q = torch.empty((out_rows, out_cols), dtype=torch.uint8, device=x.device)
    s = scale_inv if scale_inv is not None else colmajor_grid(out_rows, (out_cols + 127) // 128, x.device)
    ld_s = _grid_ld(s, out_rows)
    if rule == SCALE_RULE_FP32:
        _check("fp8_quant_1x128", lib().fp8_quant_1x128(x.data_ptr(), xt, rows, cols, _ld(x), q.data_ptr(),
                                                        q.stride(0), s.data_ptr(), ld_s, int(transpose_out),
                                                        _stream(x)))
    else:
        _check("fp8_quant_1x128_ex", lib().fp8_quant_1x128_ex(x.data_ptr(), xt, rows, cols, _ld(x), q.data_ptr(),
                                                              q.stride(0), s.data_ptr(), ld_s, int(transpose_out),
                                                              int(rule), _stream(x)))
    return q, s


def fp8_quant_1x128_dual(x: torch.Tensor, out=None, rule: int = SCALE_RULE_FP32):
    """Both 1x128 quantizations from one read of x: returns (q, scale_inv,
    q_t, scale_inv_t), equal to fp8_quant_1x128(x) followed by
    fp8_quant_1x128(x, transpose_out=True).  Preallocated outputs may be
    passed as out=(q, scale_inv, q_t, scale_inv_t).  rule as fp8_quant_1x128."""
    rows, cols = x.shape
    xt = _dtype_code(x)
    if out is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        s = colmajor_grid(rows, (cols + 127) // 128, x.device)
        qt = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
        st = colmajor_grid(cols, (rows + 127) // 128, x.device)
    else:
        q, s, qt, st = out
    args = (x.data_ptr(), xt, rows, cols, _ld(x), q.data_ptr(), q.stride(0), s.data_ptr(), _grid_ld(s, rows),
            qt.data_ptr(), qt.stride(0), st.data_ptr(), _grid_ld(st, cols))
    if rule == SCALE_RULE_FP32:
        _check("fp8_quant_1x128_dual", lib().fp8_quant_1x128_dual(*args, _stream(x)))
    else:
        _check("fp8_quant_1x128_dual_ex", lib().fp8_quant_1x128_dual_ex(*args, int(rule), _stream(x)))
    return q, s, qt, st


def fp8_quant_128x128(x: torch.Tensor, want_q: bool = True, want_qt: bool = False, out=None,
                      rule: int = SCALE_RULE_FP32):
    """Returns (q, scale_inv, q_t, scale_inv_t); the unrequested pair is None.
    q: rows x cols, grid ceil(rows/128) x ceil(cols/128).  q_t: cols x rows
    (the same quantized tiles transposed), grid ceil(cols/128) x ceil(rows/128).
    Preallocated outputs may be passed as out=(q, s, q_t, s_t).  rule as
    fp8_quant_1x128."""
    rows, cols = x.shape
    xt = _dtype_code(x)
    rb, cb = (rows + 127) // 128, (cols + 127) // 128
    q = s = qt = st = None
    if out is not None:
        q, s, qt, st = out
    qp = sp = qtp = stp = 0
    ldq = lds = ldqt = ldst = 0
    if want_q:
        if q is None:
            q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
            s = colmajor_grid(rb, cb, x.device)
        qp, sp, ldq, lds = q.data_ptr(), s.data_ptr(), q.stride(0), _grid_ld(s, rb)
    if want_qt:
        if qt is None:
            qt = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
            st = colmajor_grid(cb, rb, x.device)
        qtp, stp, ldqt, ldst = qt.data_ptr(), st.data_ptr(), qt.stride(0), _grid_ld(st, cb)
    args = (x.data_ptr(), xt, rows, cols, _ld(x), qp, ldq, sp, lds, qtp, ldqt, stp, ldst)
    if rule == SCALE_RULE_FP32:
        _check("fp8_quant_128x128", lib().fp8_quant_128x128(*args, _stream(x)))
    else:
        _check("fp8_quant_128x128_ex", lib().fp8_quant_128x128_ex(*args, int(rule), _stream(x)))
    return q, s, qt, st


def fp8_quant_tensor(x: torch.Tensor, workspace: Optional[torch.Tensor] = None):
    """Returns (q, scale_inv[1])."""
    n = x.numel()
    xc = x.contiguous()
    xt = _dtype_code(x)
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((1,), dtype=torch.float32, device=x.device)
    wsb = lib().fp8_quant_tensor_workspace_size(n)
    if workspace is None:
        workspace = torch.empty((wsb,), dtype=torch.uint8, device=x.device)
    _check("fp8_quant_tensor", lib().fp8_quant_tensor(xc.data_ptr(), xt, n, q.data_ptr(), s.data_ptr(),
                                                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                                      _stream(x)))
    return q, s


def fp8_quant_rowwise(x: torch.Tensor):
    """Returns (q, scale_inv[rows])."""
    rows, cols = x.shape
    xt = _dtype_code(x)
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    s = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _check("fp8_quant_rowwise", lib().fp8_quant_rowwise(x.data_ptr(), xt, rows, cols, _ld(x), q.data_ptr(),
                                                        q.stride(0), s.data_ptr(), _stream(x)))
    return q, s


# ---------------------------------------------------------------------------- GEMM
def fp8_scaled_gemm_workspace_size(M: int, N: int, K: int, mode: int) -> int:
    return int(lib().fp8_scaled_gemm_workspace_size(M, N, K, mode))


def fp8_scaled_gemm(A: torch.Tensor, Bt: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor, mode: int,
                    out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, split_k: bool = True) -> torch.Tensor:
    """D = scaled(A . Bt^T).  A: M x K uint8 (e4m3), Bt: N x K uint8 (e4m3).
    Scales as returned by the quantization functions (TENSOR: 1 element;
    ROWWISE: M / N elements; BLOCK: column-major grids)."""
    M, K = A.shape
    N, K2 = Bt.shape
    if K2 != K:
        raise ValueError("A and Bt must share K")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    oc = F32 if out.dtype == torch.float32 else BF16
    if mode in BLOCK_MODES:
        ld_sa = _grid_ld(scale_a, M)
        ld_sb = _grid_ld(scale_b, scale_b.shape[0])
    else:
        ld_sa = ld_sb = 0
    wsb = fp8_scaled_gemm_workspace_size(M, N, K, mode) if split_k else 0
    if wsb > 0 and workspace is None:
        workspace = torch.empty((wsb,), dtype=torch.uint8, device=A.device)
    wp = workspace.data_ptr() if (workspace is not None and wsb > 0) else 0
    wn = workspace.numel() * workspace.element_size() if (workspace is not None and wsb > 0) else 0
    _check("fp8_scaled_gemm", lib().fp8_scaled_gemm(M, N, K, A.data_ptr(), _ld(A), Bt.data_ptr(), _ld(Bt),
                                                    scale_a.data_ptr(), ld_sa, scale_b.data_ptr(), ld_sb, mode,
                                                    SCALE_COL_MAJOR, out.data_ptr(), _ld(out), oc, wp, wn,
                                                    _stream(A)))
    return out


def fp8_scaled_gemm_ex(A: torch.Tensor, B: torch.Tensor, b_major: int, scale_a: torch.Tensor,
                       scale_b: torch.Tensor, mode: int, out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       split_k: bool = True) -> torch.Tensor:
    """D = scaled(A . B).  A: M x K uint8 (e4m3).  b_major = MAJOR_MN: B is the
    K x N uint8 matrix itself (N contiguous), with a TENSOR / ROWWISE scale or
    the ceil(K/128) x ceil(N/128) grid fp8_quant_128x128 writes for it;
    b_major = MAJOR_K: B is B^T (N x K), exactly fp8_scaled_gemm."""
    if b_major == MAJOR_K:
        return fp8_scaled_gemm(A, B, scale_a, scale_b, mode, out_dtype=out_dtype, out=out, workspace=workspace,
                               split_k=split_k)
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError("A (M x K) and B (K x N) must share K")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    oc = F32 if out.dtype == torch.float32 else BF16
    if mode in BLOCK_MODES:
        ld_sa = _grid_ld(scale_a, M)
        ld_sb = _grid_ld(scale_b, scale_b.shape[0])
    else:
        ld_sa = ld_sb = 0
    wsb = fp8_scaled_gemm_workspace_size(M, N, K, mode) if split_k else 0
    if wsb > 0 and workspace is None:
        workspace = torch.empty((wsb,), dtype=torch.uint8, device=A.device)
    wp = workspace.data_ptr() if (workspace is not None and wsb > 0) else 0
    wn = workspace.numel() * workspace.element_size() if (workspace is not None and wsb > 0) else 0
    _check("fp8_scaled_gemm_ex", lib().fp8_scaled_gemm_ex(M, N, K, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B),
                                                          b_major, scale_a.data_ptr(), ld_sa, scale_b.data_ptr(),
                                                          ld_sb, mode, SCALE_COL_MAJOR, out.data_ptr(), _ld(out),
                                                          oc, wp, wn, _stream(A)))
    return out


def grouped_scale_grids(groups: int, N: int, K: int, device) -> torch.Tensor:
    """Allocate the stacked 128x128 scale grids of a grouped GEMM's B: a
    (groups, ceil(K/128), ld) fp32 tensor, ld = ceil(N/128) rounded up to 4.
    grouped_grid_view(t, g, N) is group g's (ceil(N/128) x ceil(K/128))
    column-major grid, the form fp8_quant_128x128 fills (out=...)."""
    nb, kb = (N + 127) // 128, (K + 127) // 128
    return torch.empty((groups, kb, _round_up(nb, 4)), dtype=torch.float32, device=device)


def grouped_grid_view(t: torch.Tensor, g: int, N: int) -> torch.Tensor:
    """Group g's grid of a grouped_scale_grids tensor: ceil(N/128) x ceil(K/128),
    column-major (strides (1, ld))."""
    return t[g][:, :(N + 127) // 128].t()


def fp8_scaled_gemm_grouped(A: torch.Tensor, Bt: torch.Tensor, group_rows, scale_a: torch.Tensor,
                            scale_b: torch.Tensor, N: int, out_dtype: torch.dtype = torch.bfloat16,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped 1x128 x 128x128 GEMM: for each group g, rows of A from
    sum(group_rows[:g]) on (group_rows[g] of them) times B_g^T = rows
    g*N .. g*N+N-1 of Bt.  A: (sum rows) x K uint8; Bt: (G*N) x K uint8;
    scale_a: the 1x128 grid over A's rows; scale_b: grouped_scale_grids(G, N, K).
    Returns D (sum rows) x N."""
    rows = [int(r) for r in group_rows]
    G = len(rows)
    Mt, K = A.shape
    if Mt != sum(rows) or Bt.shape != (G * N, K):
        raise ValueError("A must hold sum(group_rows) rows and Bt G*N rows of K bytes")
    if scale_b.dim() != 3 or scale_b.dtype != torch.float32 or not scale_b.is_contiguous() or scale_b.shape[0] != G:
        raise ValueError("scale_b must be grouped_scale_grids(G, N, K)")
    if out is None:
        out = torch.empty((Mt, N), dtype=out_dtype, device=A.device)
    oc = F32 if out.dtype == torch.float32 else BF16
    gr = (ctypes.c_int64 * G)(*rows)
    ld_sa = _grid_ld(scale_a, max(Mt, 1))
    _check("fp8_scaled_gemm_grouped",
           lib().fp8_scaled_gemm_grouped(G, ctypes.cast(gr, ctypes.c_void_p), N, K, A.data_ptr(), _ld(A), Bt.data_ptr(),
                                         _ld(Bt), scale_a.data_ptr(), ld_sa, scale_b.data_ptr(), scale_b.shape[2],
                                         scale_b.shape[1] * scale_b.shape[2], SCALE_BLOCK_1x128_128x128,
                                         SCALE_COL_MAJOR, out.data_ptr(), _ld(out), oc, _stream(A)))
    return out


def fp8_scaled_gemm_quant(A: torch.Tensor, Bt: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor, mode: int,
                          out: Optional[torch.Tensor] = None, store_out: bool = True,
                          q_out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None):
    """D = scaled(A . Bt^T) in bf16, quantized 1x128 along N in the GEMM's
    epilogue: returns (D or None, q uint8 M x N, scale_inv grid M x ceil(N/128)),
    byte-identical to fp8_quant_1x128(D).  store_out=False skips writing D."""
    M, K = A.shape
    N, K2 = Bt.shape
    if K2 != K:
        raise ValueError("A and Bt must share K")
    if store_out and out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    if not store_out:
        out = None
    if q_out is None:
        # the byte rows start 16-byte aligned (pitch rounded up to 16)
        q_out = torch.empty((M, (N + 15) // 16 * 16), dtype=torch.uint8, device=A.device)[:, :N]
    if scale_out is None:
        scale_out = colmajor_grid(M, (N + 127) // 128, A.device)
    if mode == SCALE_BLOCK_1x128_128x128:
        ld_sa = _grid_ld(scale_a, M)
        ld_sb = _grid_ld(scale_b, scale_b.shape[0])
    else:
        ld_sa = ld_sb = 0
    dp, ldd = (out.data_ptr(), _ld(out)) if out is not None else (0, 0)
    _check("fp8_scaled_gemm_quant",
           lib().fp8_scaled_gemm_quant(M, N, K, A.data_ptr(), _ld(A), Bt.data_ptr(), _ld(Bt), scale_a.data_ptr(),
                                       ld_sa, scale_b.data_ptr(), ld_sb, mode, SCALE_COL_MAJOR, dp, ldd,
                                       q_out.data_ptr(), q_out.stride(0), scale_out.data_ptr(),
                                       _grid_ld(scale_out, M), _stream(A)))
    return out, q_out, scale_out


# ---------------------------------------------------------------------------- norm and 4-bit helpers
_native = None


def _load_native():
    """The extension module that checks the arguments of the functions below and calls the library (csrc/binding.cpp)."""
    global _native
    lib()
    path = _build.binding_path()
    if not os.path.exists(path):
        raise ImportError(f"the extension module is not built ({path}); run fp8_block_scaled_11_b200/build.py")
    spec = importlib.util.spec_from_file_location(f"{__package__}._binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _native = module
    return _native


def _index(device) -> int:
    """The index of a CUDA device (-1: the current one, or no CUDA device): a workspace is sized for the device it is
    allocated on."""
    if device is None:
        return -1
    d = device if isinstance(device, torch.device) else torch.device(device)
    return d.index if d.type == "cuda" and d.index is not None else -1


# ---------------------------------------------------------------------------- microscaled 4 bits
def fp4_scale_tiles(rows: int, cols: int, device) -> torch.Tensor:
    """Allocate the scale tiles of a rows x cols matrix of 4-bit codes: a uint8
    tensor (ceil(rows/128), ceil(cols/128), 32, 4, 4) whose element [i//128,
    g//4, i%32, i//32%4, g%4] is the scale byte of row i, group g (32 columns)."""
    return torch.empty(((rows + 127) // 128, (cols + 127) // 128, 32, 4, 4), dtype=torch.uint8, device=device)


def _packed(rows: int, cols: int, device) -> torch.Tensor:
    """rows x cols/2 bytes of packed codes whose rows start 16-byte aligned."""
    return torch.empty((rows, _round_up(cols // 2, 16)), dtype=torch.uint8, device=device)[:, :cols // 2]


def fp4_quant_1x32(x: torch.Tensor, transpose_out: bool = False, q: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None):
    """Microscaled 4-bit quantization: returns (q uint8 rows x cols/2, scale
    tiles).  transpose_out=False: groups of 32 along the columns of x (cols %
    32 == 0).  transpose_out=True: groups along its rows (rows % 32 == 0); q is
    cols x rows/2.  Preallocated outputs may be passed as q / scale."""
    if q is None or scale is None:
        rows, cols = x.shape
        if transpose_out:
            rows, cols = cols, rows
        q = _packed(rows, cols, x.device) if q is None else q
        scale = fp4_scale_tiles(rows, cols, x.device) if scale is None else scale
    status = (_native or _load_native()).quant(x, transpose_out, q, scale)
    if status:
        raise Fp8bsError("fp4_quant_1x32", status)
    return q, scale


def fp4_dequant_1x32(q: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of packed 4-bit codes and their scale tiles."""
    if out is None:
        out = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=out_dtype, device=q.device)
    status = (_native or _load_native()).dequant(q, scale, out)
    if status:
        raise Fp8bsError("fp4_dequant_1x32", status)
    return out


def fp4_scaled_gemm_workspace(M: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """Allocate the split-K workspace of a product of these sizes (None where it needs none)."""
    n = (_native or _load_native()).product_workspace(M, N, K, _index(device))
    return torch.empty((n,), dtype=torch.uint8, device=device) if n else None


def fp4_scaled_gemm(A: torch.Tensor, Bt: torch.Tensor, scale_a: torch.Tensor, scale_b: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, split_k: bool = True) -> torch.Tensor:
    """D = A . Bt^T of two microscaled 4-bit matrices: A M x K/2 and Bt N x K/2
    uint8 (two codes a byte) with their scale tiles, as fp4_quant_1x32 returns
    them.  D: M x N, bf16 or fp32."""
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=out_dtype, device=A.device)
    if not split_k:
        workspace = None
    elif workspace is None:
        M, half = A.shape
        workspace = fp4_scaled_gemm_workspace(M, Bt.shape[0], 2 * half, A.device)
    status = (_native or _load_native()).product(A, Bt, scale_a, scale_b, out, workspace)
    if status:
        raise Fp8bsError("fp4_scaled_gemm", status)
    return out


# ---------------------------------------------------------------------------- RMS norm
def rmsnorm_quant_buffers(x: torch.Tensor, residual: bool = False, want_y: bool = False, bits: int = 8):
    """Allocate the outputs of fp8_rmsnorm_quant_1x128 (bits = 8) or
    fp4_rmsnorm_quant_1x32 (bits = 4) for inputs like x: (q, scale, h, rstd, y),
    h and y None where they are not asked for."""
    rows, cols = x.shape
    dev = x.device
    if bits == 8:
        q, s = (torch.empty((rows, cols), dtype=torch.uint8, device=dev),
                colmajor_grid(rows, (cols + 127) // 128, dev))
    elif bits == 4:
        q, s = _packed(rows, cols, dev), fp4_scale_tiles(rows, cols, dev)
    else:
        raise ValueError("bits is 8 or 4")
    return (q, s, torch.empty((rows, cols), dtype=x.dtype, device=dev) if residual else None,
            torch.empty((rows,), dtype=torch.float32, device=dev),
            torch.empty((rows, cols), dtype=x.dtype, device=dev) if want_y else None)


def fp8_rmsnorm_quant_1x128(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, want_y: bool = False, out=None, rule: int = SCALE_RULE_FP32):
    """RMS norm of h = x + residual with its result quantized 1x128 in e4m3:
    returns (q, scale_inv grid, h, rstd, y); h is x without a residual, y (the
    norm's value in x's dtype) None unless want_y.  Preallocated outputs may be
    passed as out (rmsnorm_quant_buffers); h may be x or residual itself."""
    if out is None:
        out = rmsnorm_quant_buffers(x, residual is not None, want_y)
    q, s, h, rstd, y = out
    status = (_native or _load_native()).norm(8, rule, x, weight, residual, eps, q, s, h, rstd, y)
    if status:
        raise Fp8bsError("fp8_rmsnorm_quant_1x128", status)
    return q, s, x if residual is None else h, rstd, y


def fp4_rmsnorm_quant_1x32(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, want_y: bool = False, out=None):
    """fp8_rmsnorm_quant_1x128 with its result in microscaled 4 bits: q is rows x
    cols/2 packed codes, the scales are scale tiles (bits=4 buffers)."""
    if out is None:
        out = rmsnorm_quant_buffers(x, residual is not None, want_y, 4)
    q, s, h, rstd, y = out
    status = (_native or _load_native()).norm(4, 0, x, weight, residual, eps, q, s, h, rstd, y)
    if status:
        raise Fp8bsError("fp4_rmsnorm_quant_1x32", status)
    return q, s, x if residual is None else h, rstd, y


def rmsnorm_backward_workspace(h: torch.Tensor) -> torch.Tensor:
    """Allocate the workspace of fp8bs_rmsnorm_backward for inputs like h."""
    n = (_native or _load_native()).norm_backward_workspace(h.shape[0], h.shape[1], _index(h.device))
    return torch.empty((n,), dtype=torch.uint8, device=h.device)


def fp8bs_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                           dh: Optional[torch.Tensor] = None, out=None, workspace: Optional[torch.Tensor] = None):
    """Gradients of the norm: returns (dx, dweight fp32) from dy (the gradient of
    y), the forward pass's h and rstd, and dh (the gradient that reaches h past
    the norm; added to dx).  Preallocated outputs may be passed as out=(dx,
    dweight); dx may be dy, dh or h itself."""
    dx, dw = out if out is not None else (torch.empty(h.shape, dtype=h.dtype, device=h.device),
                                          torch.empty((h.shape[1],), dtype=torch.float32, device=h.device))
    if workspace is None:
        workspace = rmsnorm_backward_workspace(h)
    status = (_native or _load_native()).norm_backward(dy, h, weight, rstd, dh, dx, dw, workspace)
    if status:
        raise Fp8bsError("fp8bs_rmsnorm_backward", status)
    return dx, dw


def fp8bs_status_string(status: int) -> str:
    return lib().fp8bs_status_string(status).decode()


def fp8bs_check_device_error(stream: Optional[torch.cuda.Stream] = None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(lib().fp8bs_check_device_error(ctypes.c_void_p(s.cuda_stream)))


def fp8_quant_tensor_noalloc(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                             scale_inv: Optional[torch.Tensor] = None):
    """Per-tensor quantization through fp8_quant_tensor_noalloc (no workspace:
    the library uses its built-in 16 KB scratch).  Returns (q, scale_inv[1]);
    pass preallocated q / scale_inv to keep the call itself allocation-free.

    The call cannot copy (a copy would allocate), so x must already be a
    contiguous bf16 / fp32 tensor on the current CUDA device; q must be a
    contiguous uint8 tensor with as many elements as x and scale_inv a
    contiguous fp32 tensor with at least one element, on the same device.
    Anything else raises ValueError before the library is called."""
    dev = torch.device("cuda", torch.cuda.current_device())
    if x.device != dev or not x.is_contiguous():
        raise ValueError("fp8_quant_tensor_noalloc: x must be contiguous and on the current CUDA device")
    xt = _dtype_code(x)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale_inv is None:
        scale_inv = torch.empty((1,), dtype=torch.float32, device=x.device)
    if q.dtype != torch.uint8 or q.numel() != x.numel() or not q.is_contiguous() or q.device != dev:
        raise ValueError("fp8_quant_tensor_noalloc: q must be a contiguous uint8 tensor of x.numel() elements "
                         "on the current CUDA device")
    if (scale_inv.dtype != torch.float32 or scale_inv.numel() < 1 or not scale_inv.is_contiguous()
            or scale_inv.device != dev):
        raise ValueError("fp8_quant_tensor_noalloc: scale_inv must be a contiguous fp32 tensor with at least "
                         "one element on the current CUDA device")
    _check("fp8_quant_tensor_noalloc", lib().fp8_quant_tensor_noalloc(x.data_ptr(), xt, x.numel(), q.data_ptr(),
                                                                      scale_inv.data_ptr(), _stream(x)))
    return q, scale_inv
