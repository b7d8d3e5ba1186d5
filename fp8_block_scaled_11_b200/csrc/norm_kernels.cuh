// norm_kernels.cuh -- root-mean-square norm with the residual's addition and its
// result quantised, and the norm's backward pass.
//
//   forward   h = round(x + residual) to x's type (h = x without a residual);
//             rstd = 1 / sqrt(mean_j h_j^2 + eps); y = h * rstd * w, in fp32;
//             y is quantised straight from fp32: 1x128 groups in e4m3, or groups
//             of 32 in microscaled 4 bits, by the rules of quant_kernels.cuh and
//             mx4.cuh.
//   backward  n = h * rstd; g = dy * w;
//             dx = rstd * (g - n * mean_j(g_j n_j)) + dh;   dw = sum_rows dy * n.
//
// All sums are fp32, each in an order that the sizes and the device fix.  Both
// passes are bound by memory: the forward reads x and the residual and writes h
// and the codes once, the backward reads dy, h and dh and writes dx once.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "mx4.cuh"
#include "quant_kernels.cuh"
#include "fp4_quant_kernels.cuh"

namespace fp8bs {

struct NormParams {
    const void* x;
    const void* res;            // nullptr: no residual
    const void* w;
    void* h;                    // written when there is a residual
    float* rstd;                // nullable
    void* y;                    // nullable, x's type
    uint8_t* q;
    void* scale;                // fp32 grid (8 bits) or scale tiles (4 bits)
    int64_t rows, cols, ldx, ldr, ldh, ldy, ldq;
    int64_t lds;                // leading dimension of the fp32 grid, or scale tiles per row block
    float eps;
    int w_f32, pow2;
};

// Eight weights as fp32 (bf16 or fp32 in memory).
__device__ __forceinline__ void load_weight8(const void* w, int w_f32, int64_t c, float (&f)[8])
{
    if (w_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        Vec8<__nv_bfloat16> v;
        v.raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c));
        v.get(f);
    }
}

// Eight fp32 values rounded to T, stored (16-byte stores).
__device__ __forceinline__ void store8(float* p, const float (&f)[8])
{
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                                              cvt_bf16x2(f[6], f[7]));
}

// f rounded to T's precision, in place.
template <typename T>
__device__ __forceinline__ void round8(float (&f)[8])
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = cvt_bf16x2(f[2 * i], f[2 * i + 1]);
            f[2 * i] = __uint_as_float(p << 16);
            f[2 * i + 1] = __uint_as_float(p & 0xFFFF0000u);
        }
    }
}

// Sum over the blockDim.x threads of this row (blockDim.x a multiple of 32; all
// threads of the CTA take part).  `part` holds one float per warp of the CTA.
__device__ __forceinline__ float row_sum(float v, float* part)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float* mine = part + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += mine[i];
    return s;
}

// Eight normalised values y of row r, columns c .. c+7 (zero past the last
// column): quantised and stored with their group's scale.  Called by whole
// warps, lane l holding the l-th eight columns of 256.
template <int BITS>
__device__ __forceinline__ void quantise_store(const NormParams& p, int64_t r, int64_t c, bool ok, const float (&y)[8])
{
    const int lane = threadIdx.x & 31;
    if constexpr (BITS == 8) {
        float m = absmax8(y);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = p.pow2 ? scale_rule<true>(m) : scale_rule<false>(m);
        if (ok) {
            *reinterpret_cast<uint2*>(p.q + r * p.ldq + c) = quant8(y, s);
            if ((lane & 15) == 0) static_cast<float*>(p.scale)[r + (c >> 7) * p.lds] = __frcp_rn(s);
        }
    } else {
        const uint32_t byte = mx4_scale_byte(group32_absmax(y));
        const uint32_t codes = mx4_pack8(y, mx4_inv_scale(byte));
        const uint32_t word = sf_gather_word(ok ? byte : 127u, lane);
        if (ok) {
            *reinterpret_cast<uint32_t*>(p.q + r * p.ldq + (c >> 1)) = codes;
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.scale) + sf_word_offset(r, c >> 7, p.lds)) = word;
        }
    }
}

// --------------------------------------------------------------------------
// Forward, rows of at most 8 * VPT * blockDim.x columns: a row's values stay in
// registers between the sum of squares and the quantisation, so memory is read
// once.  Row blockIdx.x * blockDim.y + threadIdx.y; thread t holds the eights
// t, t + blockDim.x, ... of the row, so that 16 neighbouring lanes hold a group
// of 128.
// --------------------------------------------------------------------------
template <typename T, int BITS, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rmsnorm_quant_kernel(const NormParams p)
{
    __shared__ float part[32];
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool row_ok = r < p.rows;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* res = static_cast<const T*>(p.res) + r * p.ldr;
    float v[VPT][8];
    {
        Vec8<T> a[VPT], b[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
            const bool ok = row_ok && c < p.cols;
            a[i].zero();
            b[i].zero();
            if (ok) a[i].load(x + c);
            if (ok && p.res != nullptr) b[i].load(res + c);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
            a[i].get(v[i]);
            if (p.res != nullptr) {
                float f[8];
                b[i].get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += f[j];
                round8<T>(v[i]);
                if (row_ok && c < p.cols) store8(static_cast<T*>(p.h) + r * p.ldh + c, v[i]);
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    ss = row_sum(ss, part);
    const float rstd = __frcp_rn(__fsqrt_rn(ss / (float)p.cols + p.eps));
    if (row_ok && threadIdx.x == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
        const bool ok = row_ok && c < p.cols;
        float y[8];
        if (ok) {
            load_weight8(p.w, p.w_f32, c, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= v[i][j] * rstd;
            if (p.y != nullptr) store8(static_cast<T*>(p.y) + r * p.ldy + c, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.f;
        }
        quantise_store<BITS>(p, r, c, ok, y);
    }
}

// --------------------------------------------------------------------------
// Forward, rows of any width: one CTA per row goes over it twice and takes the
// second look at h from memory (the caches, mostly).
// --------------------------------------------------------------------------
template <typename T, int BITS>
__global__ void __launch_bounds__(512) rmsnorm_quant_wide_kernel(const NormParams p)
{
    __shared__ float part[32];
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* res = static_cast<const T*>(p.res) + r * p.ldr;
    T* h = static_cast<T*>(p.h) + r * p.ldh;
    float ss = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.cols; c += (int64_t)blockDim.x * 8) {
        Vec8<T> a;
        float v[8];
        a.load(x + c);
        a.get(v);
        if (p.res != nullptr) {
            float f[8];
            a.load(res + c);
            a.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
            round8<T>(v);
            store8(h + c, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
    }
    ss = row_sum(ss, part);
    const float rstd = __frcp_rn(__fsqrt_rn(ss / (float)p.cols + p.eps));
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    // each thread reads back what it wrote itself
    const T* src = p.res != nullptr ? h : x;
    const int64_t top = (p.cols + 255) / 256 * 256;       // whole warps take part in the groups' maxima
    for (int64_t c = (int64_t)threadIdx.x * 8; c < top; c += (int64_t)blockDim.x * 8) {
        const bool ok = c < p.cols;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        if (ok) {
            Vec8<T> a;
            float v[8];
            a.load(src + c);
            a.get(v);
            load_weight8(p.w, p.w_f32, c, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= v[j] * rstd;
            if (p.y != nullptr) store8(static_cast<T*>(p.y) + r * p.ldy + c, y);
        }
        quantise_store<BITS>(p, r, c, ok, y);
    }
}

// --------------------------------------------------------------------------
// Backward
// --------------------------------------------------------------------------
struct NormBackParams {
    const void* dy;
    const void* h;
    const void* dh;             // nullptr: no gradient beside the norm's
    const void* w;
    const float* rstd;
    void* dx;
    float* part;                // [parts][cols] partial sums of dw
    float* dot;                 // [rows] mean(g n) (wide rows only)
    int64_t rows, cols, lddy, ldh, lddh, lddx;
    int w_f32;
};

// Rows of at most 8 * VPT * blockDim.x columns: a CTA goes over rows blockIdx.x
// * blockDim.y + threadIdx.y, + gridDim.x * blockDim.y, ...; a thread keeps its
// columns' weights and sums of dw in registers over all of them and leaves the
// sums in row blockIdx.x * blockDim.y + threadIdx.y of `part`.
template <typename T, int VPT>
__global__ void __launch_bounds__(512) rmsnorm_back_kernel(const NormBackParams p)
{
    __shared__ float part[2][16];
    float w[VPT][8], dw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = 0.f;
        if (c < p.cols) load_weight8(p.w, p.w_f32, c, w[i]);
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const float inv = 1.f / (float)p.cols;
    int flip = 0;
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < p.rows; base += step, flip ^= 1) {
        const int64_t r = base + threadIdx.y;
        const bool row_ok = r < p.rows;
        const float rstd = row_ok ? p.rstd[r] : 0.f;
        Vec8<T> a[VPT], b[VPT], d[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
            const bool ok = row_ok && c < p.cols;
            a[i].zero();
            b[i].zero();
            d[i].zero();
            if (ok) a[i].load(static_cast<const T*>(p.dy) + r * p.lddy + c);
            if (ok) b[i].load(static_cast<const T*>(p.h) + r * p.ldh + c);
            if (ok && p.dh != nullptr) d[i].load(static_cast<const T*>(p.dh) + r * p.lddh + c);
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float dy[8], n[8];
            a[i].get(dy);
            b[i].get(n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[j] *= rstd;
                const float t = dy[j] * n[j];
                dw[i][j] += t;
                dot += t * w[i][j];
            }
        }
        // two sets of partial sums: a warp may be a row ahead of the slowest one
        dot = row_sum(dot, part[flip]) * inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
            if (row_ok && c < p.cols) {
                float dy[8], n[8], f[8];
                a[i].get(dy);
                b[i].get(n);
                d[i].get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += rstd * (dy[j] * w[i][j] - n[j] * rstd * dot);
                store8(static_cast<T*>(p.dx) + r * p.lddx + c, f);
            }
        }
    }
    float* dst = p.part + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * p.cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * 8;
        if (c < p.cols) store8(dst + c, dw[i]);
    }
}

// Rows of any width, first launch: dot[r] = mean(g n).
template <typename T>
__global__ void __launch_bounds__(512) rmsnorm_back_dot_kernel(const NormBackParams p)
{
    __shared__ float part[16];
    const int64_t r = blockIdx.x;
    float dot = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.cols; c += (int64_t)blockDim.x * 8) {
        Vec8<T> a, b;
        float dy[8], h[8], w[8];
        a.load(static_cast<const T*>(p.dy) + r * p.lddy + c);
        b.load(static_cast<const T*>(p.h) + r * p.ldh + c);
        a.get(dy);
        b.get(h);
        load_weight8(p.w, p.w_f32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot += dy[j] * w[j] * h[j];
    }
    dot = row_sum(dot, part) * p.rstd[r];
    if (threadIdx.x == 0) p.dot[r] = dot / (float)p.cols;
}

// Second launch: CTA (x, y) goes over rows y, y + gridDim.y, ... of its 2048
// columns.
template <typename T>
__global__ void __launch_bounds__(256) rmsnorm_back_wide_kernel(const NormBackParams p)
{
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= p.cols) return;
    float w[8], dw[8];
    load_weight8(p.w, p.w_f32, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.f;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const float rstd = p.rstd[r], dot = p.dot[r];
        Vec8<T> a, b, d;
        a.load(static_cast<const T*>(p.dy) + r * p.lddy + c);
        b.load(static_cast<const T*>(p.h) + r * p.ldh + c);
        d.zero();
        if (p.dh != nullptr) d.load(static_cast<const T*>(p.dh) + r * p.lddh + c);
        float dy[8], n[8], f[8];
        a.get(dy);
        b.get(n);
        d.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            n[j] *= rstd;
            dw[j] += dy[j] * n[j];
            f[j] += rstd * (dy[j] * w[j] - n[j] * dot);
        }
        store8(static_cast<T*>(p.dx) + r * p.lddx + c, f);
    }
    store8(p.part + (int64_t)blockIdx.y * p.cols + c, dw);
}

// dw[c] = sum over the parts, 32 columns a CTA: warp w adds parts w, w + 8, ...,
// the warps' sums are added in order.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int64_t cols,
                                                         float* __restrict__ dw)
{
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < cols)
        for (int i = warp; i < parts; i += 8) sum += part[i * cols + c];
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = s[0][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) t += s[i][lane];
        dw[c] = t;
    }
}

}  // namespace fp8bs
