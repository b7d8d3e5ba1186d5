"""Plain 64-bit forms of the RMS norm, its backward pass, microscaled 4-bit
quantization and the 4-bit product (CPU, numpy/torch float64): what the GPU
tests compare the kernels with."""
import numpy as np
import torch

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LEAST = 1e-12


def scale_exponent(amax):
    """e with r = 2^e the smallest power of two such that max(amax, 1e-12) <= 6 r."""
    a = np.maximum(np.asarray(amax, dtype=np.float64), np.float64(np.float32(LEAST)))
    m, e = np.frexp(a / 6.0)                 # a / 6 = m 2^e, 0.5 <= m < 1
    e = np.where(m == 0.5, e - 1, e)
    # a / 6 is rounded: settle the border by the exact products
    e = np.where(a <= 6.0 * np.ldexp(1.0, e - 1), e - 1, e)
    return np.where(a > 6.0 * np.ldexp(1.0, e), e + 1, e)


def nearest_code(t):
    """E2M1 code of t (|t| <= 6 after rounding): nearest, ties to the even code, sign in bit 3."""
    a = np.abs(t)
    code = np.zeros(t.shape, dtype=np.uint8)
    for i in range(1, 8):
        mid = (CODES[i - 1] + CODES[i]) / 2
        code += (a > mid) if i % 2 else (a >= mid)      # a tie goes to the even one of i - 1, i
    return code | (np.signbit(t).astype(np.uint8) << 3)


def quant(x):
    """x float64 rows x cols -> (codes rows x cols, biased exponents rows x cols/32)."""
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    e = scale_exponent(np.abs(g).max(2))
    code = nearest_code(np.ldexp(g, -e[:, :, None]))
    return code.reshape(rows, cols), (e + 127).astype(np.uint8)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def tile_index(rows, groups):
    """Byte offsets of (row, group) in the scale tiles of a matrix with that many groups a row."""
    i = np.arange(rows)[:, None]
    g = np.arange(groups)[None, :]
    kcs = (groups + 3) // 4
    return ((i // 128) * kcs + g // 4) * 512 + (i % 32) * 16 + (i // 32 % 4) * 4 + g % 4


def tiles(exponents, fill=127):
    rows, groups = exponents.shape
    t = np.full(((rows + 127) // 128) * ((groups + 3) // 4) * 512, fill, dtype=np.uint8)
    t[tile_index(rows, groups)] = exponents
    return t


def value(code, exponents):
    mag = CODES[code & 7] * np.where(code & 8, -1.0, 1.0)
    return mag * np.repeat(np.ldexp(1.0, exponents.astype(np.int64) - 127), 32, axis=1)


def norm(x, residual, weight, eps):
    """(h in x's dtype, rstd, y) with float64 arithmetic on the rounded h."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    v = h.double()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + eps)
    return h, rstd, v * rstd[:, None] * weight.double()


def norm_backward(dy, h, weight, rstd, dh):
    dy, h, w = dy.double(), h.double(), weight.double()
    n = h * rstd.double()[:, None]
    g = dy * w
    dx = rstd.double()[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return dx if dh is None else dx + dh.double(), (dy * n).sum(0)
