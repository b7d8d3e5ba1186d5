// fp4_quant_kernels.cuh -- microscaled 4-bit quantisation along the columns or
// (transposed) along the rows, and back.  The scale rule and the layouts are in
// mx4.cuh.  Memory-bound: every input is read once with 16-byte loads.  At 16640 x
// 8192 bf16 quantising takes 53 us along the columns or the rows, the
// way back 54: 6.5, 6.5 and 6.4 TB/s (a plain copy reaches 6.5).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "mx4.cuh"
#include "ptx_fp4.cuh"
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

// Largest of VPT values each over the lanes that differ in the bits TOP, TOP / 2,
// .., 1: while more than one value is left, a step gives half of them away, so
// that VPT = 4 takes 5 shuffles over 16 lanes instead of 16.  On return a lane
// holds the maximum of value i whose bits are the lane's bits TOP (the higher
// bit of i), TOP / 2.  KEEP: NaN where one of the values is.
template <int VPT, int TOP, bool KEEP>
__device__ __forceinline__ float share_max(const float (&m)[VPT], int lane)
{
    float a;
    int o = TOP;
    if constexpr (VPT == 4) {
        const bool hi = lane & TOP, lo = lane & (TOP >> 1);
        float a0 = hi ? m[2] : m[0], a1 = hi ? m[3] : m[1];
        a0 = max_of<KEEP>(a0, __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], TOP));
        a1 = max_of<KEEP>(a1, __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], TOP));
        a = max_of<KEEP>(lo ? a1 : a0, __shfl_xor_sync(0xffffffffu, lo ? a0 : a1, TOP >> 1));
        o = TOP >> 2;
    } else if constexpr (VPT == 2) {
        const bool hi = lane & TOP;
        a = max_of<KEEP>(hi ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[1], TOP));
        o = TOP >> 1;
    } else {
        a = m[0];
    }
#pragma unroll
    for (; o >= 1; o >>= 1) a = max_of<KEEP>(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// The value index a lane holds after share_max, and the lane (of its TOP * 2
// lanes) that holds value i.
template <int VPT, int TOP>
__device__ __forceinline__ int share_index(int lane)
{
    if (VPT == 4) return ((lane & TOP) ? 2 : 0) + ((lane & (TOP >> 1)) ? 1 : 0);
    return VPT == 2 && (lane & TOP) ? 1 : 0;
}
template <int VPT, int TOP>
__device__ __forceinline__ int share_lane(int i)
{
    if (VPT == 4) return (i >> 1) * TOP + (i & 1) * (TOP >> 1);
    return VPT == 2 ? i * TOP : 0;
}

// --------------------------------------------------------------------------
// Groups along the columns.  A CTA owns a scale tile's 128 rows x 128 columns;
// half-warp h of 16 takes rows h, h + 16 (mod 32) of each of the four 32-row
// quarters, whose scale words are adjacent in the tile (16 bytes of one store).
// FULL: rows and columns are multiples of 128, nothing is tested.
// --------------------------------------------------------------------------
template <typename T, bool FULL>
__global__ void __launch_bounds__(256) fp4_quant_rows_kernel(const T* x, int64_t rows, int64_t cols,
                                                             int64_t ldx, uint8_t* q, int64_t ldq,
                                                             uint8_t* sf, int kcs)
{
    const int lane = threadIdx.x & 31;
    const int hw = threadIdx.x >> 4;
    const int rb = (int)blockIdx.x / kcs, kc = (int)blockIdx.x - rb * kcs;
    const int64_t c = (int64_t)kc * 128 + (threadIdx.x & 15) * 8;
    const bool col_ok = FULL || c < cols;       // cols % 32 == 0: a group is all in or all out
    const int64_t r0 = (int64_t)rb * 128 + hw;
    const T* src = x + r0 * ldx + c;
    uint8_t* dst = q + r0 * ldq + (c >> 1);
    uint8_t* scales = sf + ((int64_t)rb * kcs + kc) * (int64_t)kSfTileBytes + hw * 16;
    // row 16 i + 32 j past r0
    auto row_ok = [&](int i, int j) { return FULL || (col_ok && r0 + 16 * i + 32 * j < rows); };
    Vec8<T> v[2][4];
    grid_begin();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!FULL) v[i][j].zero();
            if (row_ok(i, j)) load_stream(v[i][j], src + (16 * i + 32 * j) * ldx);
        }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // lane l of a group's four takes row l's maximum: one scale a lane
        Eight e[4];
        float m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = eight_of(v[i][j]);
            m[j] = absmax<true>(e[j]);
        }
        const uint32_t mine = mx4_scale_byte(share_max<4, 2, true>(m, lane));
        const uint32_t word = sf_gather_word(col_ok ? mine : 127u, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t byte = __shfl_sync(0xffffffffu, mine, (lane & 28) + share_lane<4, 2>(j));
            if (row_ok(i, j)) *reinterpret_cast<uint32_t*>(dst + (16 * i + 32 * j) * ldq) = mx4_pack8(e[j], mx4_inv_scale(byte));
        }
        // rows past the last one keep their bytes
        const int own = share_index<4, 2>(lane);
        if ((lane & 12) == 0 && (FULL || r0 + 16 * i + 32 * own < rows))
            *reinterpret_cast<uint32_t*>(scales + 256 * i + 4 * own) = word;
    }
}

// --------------------------------------------------------------------------
// Groups along the rows; the transposed codes and their scale tiles are written
// (row c of the output is column c of x).  A CTA owns 256 rows x 64 columns of x
// (128 bytes of bf16 a row to read, 128 bytes a row of codes to write), as 8 x 8
// blocks: warp w covers rows 32 w .. + 31, i.e. one group of each column.  The
// codes pass through shared memory to leave in whole 16-byte pieces; its pieces
// are permuted by the column's strip, so that a warp's words fall into 32 banks.
// FULL: whole tiles only, nothing is tested.  Four CTAs an SM for bf16 (64 registers a
// thread, none spilt; 4096 x 4096 7.1 us, with three 8.0).
// --------------------------------------------------------------------------
constexpr int kQ4Rows = 256, kQ4Cols = 64;

// The scale bytes of a group's eight columns, whose 32 rows are in the four
// lanes that differ in bits 3 and 4.  bf16: the magnitudes are compared as
// unsigned 16-bit halves (in the order of the values, NaN above infinity), two
// columns a word; half the words are given away at each step, so that a lane
// ends with one word and two scales, which it hands back.
__device__ __forceinline__ void col_scale_bytes(const Block8x8<__nv_bfloat16>& b, uint32_t (&byte)[8], int lane)
{
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[0] = __vmaxu2(m[0], b.row[i].raw.x & 0x7FFF7FFFu);
        m[1] = __vmaxu2(m[1], b.row[i].raw.y & 0x7FFF7FFFu);
        m[2] = __vmaxu2(m[2], b.row[i].raw.z & 0x7FFF7FFFu);
        m[3] = __vmaxu2(m[3], b.row[i].raw.w & 0x7FFF7FFFu);
    }
    const bool hi = lane & 16, lo = lane & 8;
    const uint32_t a0 = __vmaxu2(hi ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 16));
    const uint32_t a1 = __vmaxu2(hi ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], 16));
    const uint32_t a = __vmaxu2(lo ? a1 : a0, __shfl_xor_sync(0xffffffffu, lo ? a0 : a1, 8));
    const uint32_t mine = mx4_scale_byte(__uint_as_float(a << 16)) | mx4_scale_byte(__uint_as_float(a & 0xFFFF0000u)) << 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t two = __shfl_sync(0xffffffffu, mine, (lane & 7) + (j >> 1) * 16 + (j & 1) * 8);
        byte[2 * j] = two & 0xFFFFu;
        byte[2 * j + 1] = two >> 16;
    }
}
__device__ __forceinline__ void col_scale_bytes(const Block8x8<float>& b, uint32_t (&byte)[8], int)
{
    float m[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        b.row[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = max_nan(m[j], fabsf(f[j]));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = max_nan(m[j], __shfl_xor_sync(0xffffffffu, m[j], 8));
        m[j] = max_nan(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        byte[j] = mx4_scale_byte(m[j]);
    }
}

template <typename T, bool FULL>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) fp4_quant_cols_kernel(const T* x, int64_t rows, int64_t cols,
                                                             int64_t ldx, uint8_t* q, int64_t ldq,
                                                             uint8_t* sf, int kcs, int tiles_c)
{
    __shared__ __align__(16) uint8_t s_q[kQ4Cols * 128];
    __shared__ __align__(16) uint8_t s_sf[kQ4Cols * 8];
    const int tr = (int)blockIdx.x / tiles_c, tc = (int)blockIdx.x - tr * tiles_c;
    const int w = threadIdx.x >> 5, strip = threadIdx.x & 7, part = (threadIdx.x >> 3) & 3;
    const int64_t r0 = (int64_t)tr * kQ4Rows + w * 32 + part * 8;
    const int64_t c0 = (int64_t)tc * kQ4Cols + strip * 8;
    const bool ok = FULL || (r0 < rows && c0 < cols);     // rows % 32 == 0, cols % 16 == 0
    Block8x8<T> b;
    const T* src = x + r0 * ldx + c0;
    grid_begin();
#pragma unroll
    for (int i = 0; i < 8; ++i, src += ldx) {
        if (!FULL) b.row[i].zero();
        if (ok) load_stream(b.row[i], src);
    }
    uint32_t bytes[8];
    col_scale_bytes(b, bytes, threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = bytes[j];
        Eight e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float g[8], h[8];
            b.row[2 * i].get(g);
            b.row[2 * i + 1].get(h);
            e.v[i] = make_float2(g[j], h[j]);
        }
        const int row = strip * 8 + j;
        *reinterpret_cast<uint32_t*>(s_q + row * 128 + ((w ^ strip) * 16) + part * 4) = mx4_pack8(e, mx4_inv_scale(byte));
        // (rows past x's last: a scale of one)
        if (part == 0) s_sf[row * 8 + w] = (uint8_t)(FULL || r0 < rows ? byte : 127u);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = (threadIdx.x >> 3) + 32 * i, piece = threadIdx.x & 7;
        const int64_t c = (int64_t)tc * kQ4Cols + row, r = (int64_t)tr * kQ4Rows + piece * 32;
        if (FULL || (c < cols && r < rows))
            *reinterpret_cast<uint4*>(q + c * ldq + (r >> 1)) =
                *reinterpret_cast<const uint4*>(s_q + row * 128 + ((piece ^ (row >> 3)) * 16));
    }
    if (threadIdx.x < 2 * kQ4Cols) {
        const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
        const int64_t c = (int64_t)tc * kQ4Cols + row, kc = (int64_t)tr * 2 + half;
        if (FULL || (c < cols && kc < kcs))
            *reinterpret_cast<uint32_t*>(sf + sf_word_offset(c, kc, kcs)) =
                *reinterpret_cast<const uint32_t*>(s_sf + row * 8 + half * 4);
    }
}

// --------------------------------------------------------------------------
// Codes and scale tiles -> values (bf16 or fp32): exact, except that a value
// outside the output type's range rounds as the type does.  The same partition as
// fp4_quant_rows_kernel: a CTA owns a scale tile.
// --------------------------------------------------------------------------
template <typename T, bool FULL>
__global__ void __launch_bounds__(256) fp4_dequant_kernel(const uint8_t* q, int64_t ldq,
                                                          const uint8_t* sf, int64_t rows, int64_t cols,
                                                          int kcs, T* out, int64_t ldo)
{
    const int hw = threadIdx.x >> 4;
    const int rb = (int)blockIdx.x / kcs, kc = (int)blockIdx.x - rb * kcs;
    const int64_t c = (int64_t)kc * 128 + (threadIdx.x & 15) * 8;
    if (!FULL && c >= cols) return;              // cols % 32 == 0: a group is all in or all out
    // bf16: a lane's eight codes make 16 bytes.  fp32: a pair of lanes takes its
    // sixteen codes four at a time in turn, so that a pair stores 32 bytes in a row.
    constexpr bool kWide = sizeof(T) == 4;
    const int odd = threadIdx.x & 1;
    const int64_t r0 = (int64_t)rb * 128 + hw;
    const uint8_t* src = q + r0 * ldq + ((kWide ? c - odd * 8 : c) >> 1);
    // the scale bytes of rows r0 + 16 i + 32 j: one 16-byte row of the tile each i
    const uint8_t* scales = sf + ((int64_t)rb * kcs + kc) * (int64_t)kSfTileBytes + hw * 16 + ((threadIdx.x >> 2) & 3);
    T* dst = out + r0 * ldo + (kWide ? c - odd * 4 : c);
    uint32_t w[8], byte[8];
    grid_begin();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int dr = 16 * (i & 1) + 32 * (i >> 1);
        if (FULL || r0 + dr < rows) {
            if constexpr (kWide) {
                const uint2 v = ld_stream_u2(src + dr * ldq);
                w[i] = __byte_perm(v.x, v.y, odd ? 0x7632 : 0x5410);
            } else {
                w[i] = ld_stream_u1(src + dr * ldq);
            }
            byte[i] = scales[256 * (i & 1) + 4 * (i >> 1)];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int dr = 16 * (i & 1) + 32 * (i >> 1);
        if (FULL || r0 + dr < rows) {
            float f[8];
            mx4_unpack8(w[i], mx4_scale_value(byte[i]), f);
            if constexpr (kWide) {
                __stcs(reinterpret_cast<float4*>(dst + dr * ldo), make_float4(f[0], f[1], f[2], f[3]));
                __stcs(reinterpret_cast<float4*>(dst + dr * ldo + 8), make_float4(f[4], f[5], f[6], f[7]));
            } else {
                __stcs(reinterpret_cast<uint4*>(dst + dr * ldo),
                       make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                                  cvt_bf16x2(f[6], f[7])));
            }
        }
    }
}

}  // namespace fp8bs
