// mx4.cuh -- microscaled 4-bit values: E2M1 codes in groups of 32 along K, each
// group with one power-of-two scale held as a biased exponent (UE8M0).
//
// The scale rule: r = the smallest power of two with max|v| <= 6 r over the
// group (max|v| taken as at least 1e-12), so that no value saturates; the code
// is v / r rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the
// even code), its highest bit the sign.  v / r is exact in fp32 (r is a power of
// two), so the code has a single rounding.  A group that holds a NaN or an
// infinity gets the format's NaN scale (255), whatever its codes.
//
// Packed matrix (rows x K): row-major, two codes to a byte, the even column in
// the low half.  Scale tiles: one 512-byte tile per 128 rows x 4 groups (128
// columns), tiles of a row block one after another along K; inside a tile the
// byte of row r, group g is at (r % 32) * 16 + (r / 32 % 4) * 4 + g % 4, which
// is the order in which the tensor cores' scale-factor copy reads it: a product
// moves whole tiles and rearranges nothing.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include "ptx.cuh"
#include "ptx_load.cuh"
#include "quant_kernels.cuh"

namespace fp8bs {

constexpr uint32_t kSfTileBytes = 512;

// The larger of a and b, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The scale's byte for a group's largest magnitude (>= 0, or NaN).
// max|v| = 1.m * 2^e fits 6 r = 1.5 * 2^2 * r: r = 2^(e - 2), or twice that
// where 1.m > 1.5 (the addition carries into the exponent then).  The floor of 1e-12 keeps the byte at 85 or more; the
// largest finite fp32 gives 253; an infinity or NaN 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(float amax)
{
    const uint32_t b = __float_as_uint(max_nan(amax, 1e-12f));
    return b >= 0x7F800000u ? 255u : ((b + 0x3FFFFFu) >> 23) - 2u;
}

// 1 / r of a scale byte in [1, 253] (255: an infinity, the codes mean nothing).
__device__ __forceinline__ float mx4_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// r of any scale byte: 2^(byte - 127) (byte 0 is subnormal in fp32), 255 is NaN.
__device__ __forceinline__ float mx4_scale_value(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : byte == 0u ? 0x400000u : byte << 23);
}

// Eight values as four fp32 pairs: the arithmetic is packed (two lanes an instruction),
// since the quantising kernels in bf16 come close to the issue rate before they
// reach the memory's.
struct Eight {
    float2 v[4];
};

// Eight values read once, or (a norm's weight) again and again.
__device__ __forceinline__ float4 as_float4(uint4 v)
{
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void load_stream(Vec8<__nv_bfloat16>& v, const __nv_bfloat16* p) { v.raw = ld_stream_u4(p); }
__device__ __forceinline__ void load_stream(Vec8<float>& v, const float* p)
{
    v.a = as_float4(ld_stream_u4(p));
    v.b = as_float4(ld_stream_u4(p + 4));
}
__device__ __forceinline__ void load_kept(Vec8<__nv_bfloat16>& v, const __nv_bfloat16* p) { v.raw = ld_u4(p); }
__device__ __forceinline__ void load_kept(Vec8<float>& v, const float* p)
{
    v.a = as_float4(ld_u4(p));
    v.b = as_float4(ld_u4(p + 4));
}

template <typename T>
__device__ __forceinline__ Eight eight_of(const Vec8<T>& a)
{
    Eight e;
    if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {a.raw.x, a.raw.y, a.raw.z, a.raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) e.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
        e.v[0] = make_float2(a.a.x, a.a.y);
        e.v[1] = make_float2(a.a.z, a.a.w);
        e.v[2] = make_float2(a.b.x, a.b.y);
        e.v[3] = make_float2(a.b.z, a.b.w);
    }
    return e;
}

__device__ __forceinline__ Eight eight_zero()
{
    Eight e;
#pragma unroll
    for (int i = 0; i < 4; ++i) e.v[i] = make_float2(0.f, 0.f);
    return e;
}

// KEEP: NaN where one of the values is, else such a value does not count.
template <bool KEEP>
__device__ __forceinline__ float max_of(float a, float b)
{
    return KEEP ? max_nan(a, b) : fmaxf(a, b);
}
template <bool KEEP>
__device__ __forceinline__ float absmax(const Eight& e)
{
    float m = fabsf(e.v[0].x);
    m = max_of<KEEP>(m, fabsf(e.v[0].y));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max_of<KEEP>(max_of<KEEP>(m, fabsf(e.v[i].x)), fabsf(e.v[i].y));
    return m;
}

// Eight values times s -> eight codes, value 0 in the lowest four bits.
__device__ __forceinline__ uint32_t mx4_pack8(const Eight& e, float s)
{
    const float2 k = make_float2(s, s);
    const float2 a = fmul2(e.v[0], k), b = fmul2(e.v[1], k), c = fmul2(e.v[2], k), d = fmul2(e.v[3], k);
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

// Eight codes -> eight values times r (exact: a code's value has two bits).
__device__ __forceinline__ void mx4_unpack8(uint32_t w, float r, float (&f)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = v.x * r;
        f[2 * i + 1] = v.y * r;
    }
}

// Byte offset of the four scale bytes (one 128-column chunk) of row r, chunk kc,
// in a matrix with `kcs` chunks per row.
__device__ __forceinline__ int64_t sf_word_offset(int64_t r, int64_t kc, int64_t kcs)
{
    return ((r >> 7) * kcs + kc) * (int64_t)kSfTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

}  // namespace fp8bs
