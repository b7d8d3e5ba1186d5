// fp4_quant_kernels.cuh -- microscaled 4-bit quantisation along the columns or
// (transposed) along the rows, and back.  The scale rule and the layouts are in
// mx4.cuh.  Memory-bound: every input is read once with 16-byte loads.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "mx4.cuh"
#include "quant_kernels.cuh"

namespace fp8bs {

// The four scale bytes of a 128-column chunk, from the byte of each group (the
// same in the group's four lanes): the word in every lane of the half-warp.
__device__ __forceinline__ uint32_t sf_gather_word(uint32_t byte, int lane)
{
    uint32_t w = byte << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    return w | __shfl_xor_sync(0xffffffffu, w, 8);
}

// Largest magnitude over the four lanes that share a group of 32 values.
__device__ __forceinline__ float group32_absmax(const float (&f)[8])
{
    float m = absmax8(f);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// --------------------------------------------------------------------------
// Groups along the columns.  A CTA owns a scale tile's 128 rows x 128 columns;
// half-warp h of 16 takes rows h, h + 16 (mod 32) of each of the four 32-row
// quarters, whose scale words are adjacent in the tile (one 16-byte store).
// --------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) fp4_quant_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                             int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                             uint8_t* __restrict__ sf, int64_t kcs)
{
    const int lane = threadIdx.x & 31;
    const int hw = threadIdx.x >> 4;
    const int64_t rb = blockIdx.x / kcs, kc = blockIdx.x - rb * kcs;
    const int64_t c = kc * 128 + (threadIdx.x & 15) * 8;
    const bool col_ok = c < cols;           // cols % 32 == 0: a group is all in or all out
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r0 = rb * 128 + hw + 16 * i;
        Vec8<T> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (col_ok && r0 + 32 * j < rows) v[j].load(x + (r0 + 32 * j) * ldx + c);
            else v[j].zero();
        }
        uint32_t word[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
            v[j].get(f);
            const uint32_t byte = mx4_scale_byte(group32_absmax(f));
            const uint32_t codes = mx4_pack8(f, mx4_inv_scale(byte));
            if (col_ok && r0 + 32 * j < rows) *reinterpret_cast<uint32_t*>(q + (r0 + 32 * j) * ldq + (c >> 1)) = codes;
            word[j] = sf_gather_word(col_ok ? byte : 127u, lane);
        }
        // rows past the last one keep their bytes
        if ((lane & 15) == 0) {
            uint8_t* dst = sf + sf_word_offset(r0, kc, kcs);
            if (r0 + 96 < rows) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r0 + 32 * j < rows) *reinterpret_cast<uint32_t*>(dst + 4 * j) = word[j];
            }
        }
    }
}

// --------------------------------------------------------------------------
// Groups along the rows; the transposed codes and their scale tiles are written
// (row c of the output is column c of x).  A CTA owns 256 rows x 64 columns of x
// (128 bytes of bf16 a row to read, 128 bytes a row of codes to write), as 8 x 8
// blocks: warp w covers rows 32 w .. + 31, i.e. one group of each column.  The
// codes pass through shared memory to leave in whole 16-byte pieces; its pieces
// are permuted by the column's strip, so that a warp's words fall into 32 banks.
// --------------------------------------------------------------------------
constexpr int kQ4Rows = 256, kQ4Cols = 64;

template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) fp4_quant_cols_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                             int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                             uint8_t* __restrict__ sf, int64_t kcs, int64_t tiles_c)
{
    __shared__ __align__(16) uint8_t s_q[kQ4Cols * 128];
    __shared__ __align__(16) uint8_t s_sf[kQ4Cols * 8];
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int w = threadIdx.x >> 5, strip = threadIdx.x & 7, part = (threadIdx.x >> 3) & 3;
    const int64_t r0 = tr * kQ4Rows + w * 32 + part * 8;
    const int64_t c0 = tc * kQ4Cols + strip * 8;
    const bool ok = r0 < rows && c0 < cols;     // rows % 32 == 0, cols % 16 == 0
    Block8x8<T> b;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (ok) b.row[i].load(x + (r0 + i) * ldx + c0);
        else b.row[i].zero();
    }
    float m[8];
    b.col_absmax(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 8));
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = mx4_scale_byte(m[j]);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float g[8];
            b.row[i].get(g);
            f[i] = g[j];
        }
        const int row = strip * 8 + j;
        *reinterpret_cast<uint32_t*>(s_q + row * 128 + ((w ^ strip) * 16) + part * 4) = mx4_pack8(f, mx4_inv_scale(byte));
        // (rows past x's last: a scale of one)
        if (part == 0) s_sf[row * 8 + w] = (uint8_t)(r0 < rows ? byte : 127u);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = (threadIdx.x >> 3) + 32 * i, piece = threadIdx.x & 7;
        const int64_t c = tc * kQ4Cols + row, r = tr * kQ4Rows + piece * 32;
        if (c < cols && r < rows)
            *reinterpret_cast<uint4*>(q + c * ldq + (r >> 1)) =
                *reinterpret_cast<const uint4*>(s_q + row * 128 + ((piece ^ (row >> 3)) * 16));
    }
    if (threadIdx.x < 2 * kQ4Cols) {
        const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
        const int64_t c = tc * kQ4Cols + row, kc = tr * 2 + half;
        if (c < cols && kc < kcs)
            *reinterpret_cast<uint32_t*>(sf + sf_word_offset(c, kc, kcs)) =
                *reinterpret_cast<const uint32_t*>(s_sf + row * 8 + half * 4);
    }
}

// --------------------------------------------------------------------------
// Codes and scale tiles -> values (bf16 or fp32): exact, except that a value
// outside the output type's range rounds as the type does.  The same partition as
// fp4_quant_rows_kernel: a CTA owns a scale tile.
// --------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                          const uint8_t* __restrict__ sf, int64_t rows, int64_t cols,
                                                          int64_t kcs, T* __restrict__ out, int64_t ldo)
{
    const int hw = threadIdx.x >> 4;
    const int64_t rb = blockIdx.x / kcs, kc = blockIdx.x - rb * kcs;
    const int64_t c = kc * 128 + (threadIdx.x & 15) * 8;
    if (c >= cols) return;                       // cols % 32 == 0: a group is all in or all out
    const int group = (threadIdx.x >> 2) & 3;
    // bf16: a lane's eight codes make 16 bytes.  fp32: a pair of lanes takes its
    // sixteen codes four at a time in turn, so that a pair stores 32 bytes in a row.
    constexpr bool kWide = sizeof(T) == 4;
    const int odd = threadIdx.x & 1;
    uint32_t w[8], byte[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = rb * 128 + hw + 16 * (i & 1) + 32 * (i >> 1);
        if (r < rows) {
            if constexpr (kWide) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(q + r * ldq + ((c - odd * 8) >> 1)));
                w[i] = __byte_perm(v.x, v.y, odd ? 0x7632 : 0x5410);
            } else {
                w[i] = __ldcs(reinterpret_cast<const uint32_t*>(q + r * ldq + (c >> 1)));
            }
            byte[i] = sf[sf_word_offset(r, kc, kcs) + group];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = rb * 128 + hw + 16 * (i & 1) + 32 * (i >> 1);
        if (r < rows) {
            float f[8];
            mx4_unpack8(w[i], mx4_scale_value(byte[i]), f);
            if constexpr (kWide) {
                T* dst = out + r * ldo + (c - odd * 4);
                __stcs(reinterpret_cast<float4*>(dst), make_float4(f[0], f[1], f[2], f[3]));
                __stcs(reinterpret_cast<float4*>(dst + 8), make_float4(f[4], f[5], f[6], f[7]));
            } else {
                __stcs(reinterpret_cast<uint4*>(out + r * ldo + c),
                       make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                                  cvt_bf16x2(f[6], f[7])));
            }
        }
    }
}

}  // namespace fp8bs
