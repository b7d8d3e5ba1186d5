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
// and the codes once, the backward reads dy, h and dh and writes dx once.  At
// 16640 x 8192 bf16 the forward with residual takes 144-147 us and the backward
// with dh 171-175, 6.5-6.7 and 6.2-6.4 TB/s (a plain copy reaches 6.5).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "mx4.cuh"
#include "ptx_fp4.cuh"
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
    float eps, inv_cols;        // inv_cols = 1 / cols
    int w_f32, pow2;
};

// a + b, rounded to T.  bf16: the packed addition rounds the exact sum once; so
// does rounding the fp32 sum (the sum of two 8-bit significands is exact in fp32,
// or else next to one of them and far from a tie).
template <typename T>
__device__ __forceinline__ void add_round(Vec8<T>& a, const Vec8<T>& b)
{
    if constexpr (sizeof(T) == 2) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&a.raw);
        const uint32_t* y = reinterpret_cast<const uint32_t*>(&b.raw);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(x[i]) : "r"(x[i]), "r"(y[i]));
    } else {
        a.a.x += b.a.x; a.a.y += b.a.y; a.a.z += b.a.z; a.a.w += b.a.w;
        a.b.x += b.b.x; a.b.y += b.b.y; a.b.z += b.b.z; a.b.w += b.b.w;
    }
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec8<T>& a)
{
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = a.raw;
    } else {
        *reinterpret_cast<float4*>(p) = a.a;
        *reinterpret_cast<float4*>(p + 4) = a.b;
    }
}

// Eight fp32 values rounded to T, stored (16-byte stores).
__device__ __forceinline__ void store8(float* p, const Eight& e)
{
    *reinterpret_cast<float4*>(p) = make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& e)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(e.v[0].x, e.v[0].y), cvt_bf16x2(e.v[1].x, e.v[1].y),
                                              cvt_bf16x2(e.v[2].x, e.v[2].y), cvt_bf16x2(e.v[3].x, e.v[3].y));
}

// Eight weights as fp32 (bf16 or fp32 in memory).
__device__ __forceinline__ Eight load_weight8(const void* w, int w_f32, int64_t c)
{
    if (w_f32) {
        Vec8<float> v;
        load_kept(v, static_cast<const float*>(w) + c);
        return eight_of(v);
    }
    Vec8<__nv_bfloat16> v;
    load_kept(v, static_cast<const __nv_bfloat16*>(w) + c);
    return eight_of(v);
}

__device__ __forceinline__ float sum_squares(const Eight& e, float acc)
{
    float2 s = make_float2(acc, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = ffma2(e.v[i], e.v[i], s);
    return s.x + s.y;
}

// 1 / sqrt(a): the hardware's approximation and one Newton step (about one
// rounding from the exact value).
__device__ __forceinline__ float rstd_of(float sum, float inv_cols, float eps)
{
    const float a = fmaf(sum, inv_cols, eps);
    const float r = rsqrtf(a);
    return r * fmaf(-0.5f * a * r, r, 1.5f);
}

// y = h * rstd * w
__device__ __forceinline__ Eight normalise(const Eight& h, float rstd, const Eight& w)
{
    const float2 k = make_float2(rstd, rstd);
    Eight y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = fmul2(fmul2(h.v[i], k), w.v[i]);
    return y;
}

// Sum of n (1 to 32) warps' partial sums, 16 bytes a load.
__device__ __forceinline__ float sum_parts(const float* part, int n)
{
    float s = 0.f;
    for (int i = 0; i < n; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(part + i);
        s += (v.x + (i + 1 < n ? v.y : 0.f)) + ((i + 2 < n ? v.z : 0.f) + (i + 3 < n ? v.w : 0.f));
    }
    return s;
}

// Sum over the blockDim.x threads of this row (16, or a multiple of 32; all
// threads of the CTA take part).
__device__ __forceinline__ float row_sum(float v)
{
    __shared__ __align__(16) float part[8][32];
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 16) return v;
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.y][threadIdx.x >> 5] = v;
    __syncthreads();
    return sum_parts(part[threadIdx.y], blockDim.x >> 5);
}

// VPT eights of normalised values of row r, columns (i tx + x) 8 .. + 7 (zero past
// the last column): quantised and stored with their groups' scales.  Whole warps
// take part; 16 neighbouring lanes (4 for the groups of 32) hold a group.
// FULL: every eight is inside the matrix.
template <int BITS, int VPT, bool FULL>
__device__ __forceinline__ void quantise_store(const NormParams& p, int64_t r, bool row_ok, int tx, int x,
                                               const Eight (&y)[VPT])
{
    auto inside = [&](int c) { return FULL || (row_ok && c < p.cols); };
    const int lane = threadIdx.x + threadIdx.y * blockDim.x & 31;
    float m[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) m[i] = absmax<BITS == 4>(y[i]);
    if constexpr (BITS == 8) {
        const float top = share_max<VPT, 8, false>(m, lane);
        const float mine = p.pow2 ? scale_rule<true>(top) : scale_rule<false>(top);
        const int mi = share_index<VPT, 8>(lane);
        const int mc = (mi * tx + (x & ~15)) * 8;               // first column of the lane's own group
        const int own = VPT == 4 ? 3 : VPT == 2 ? 7 : 15;       // one of the lanes that hold the same group
        if ((lane & own) == 0 && inside(mc)) static_cast<float*>(p.scale)[r + (mc >> 7) * p.lds] = __frcp_rn(mine);
        uint8_t* q = p.q + r * p.ldq;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float s = VPT == 1 ? mine : __shfl_sync(0xffffffffu, mine, (lane & 16) + share_lane<VPT, 8>(i));
            const int c = (i * tx + x) * 8;
            if (inside(c)) {
                const float2 k = make_float2(s, s);
                float2 t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = fmul2(y[i].v[j], k);
                const uint32_t lo = cvt_e4m3x2(t[0].x, t[0].y) | (uint32_t)cvt_e4m3x2(t[1].x, t[1].y) << 16;
                const uint32_t hi = cvt_e4m3x2(t[2].x, t[2].y) | (uint32_t)cvt_e4m3x2(t[3].x, t[3].y) << 16;
                *reinterpret_cast<uint2*>(q + c) = make_uint2(lo, hi);
            }
        }
    } else {
        const float top = share_max<VPT, 2, true>(m, lane);
        const uint32_t mine = mx4_scale_byte(top);
        const int mi = share_index<VPT, 2>(lane);
        // the chunk's word: its four groups' bytes, groups past the last column 127
        const int mc = (mi * tx + (x & ~3)) * 8;
        const uint32_t word = sf_gather_word(FULL || mc < p.cols ? mine : 127u, lane);
        const int own = VPT == 4 ? 12 : VPT == 2 ? 13 : 15;
        const int chunk = (mi * tx + (x & ~15)) * 8;
        if ((lane & own) == 0 && inside(chunk))
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.scale) + sf_word_offset(r, chunk >> 7, p.lds)) = word;
        uint8_t* q = p.q + r * p.ldq;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t byte = VPT == 1 ? mine : __shfl_sync(0xffffffffu, mine, (lane & 28) + share_lane<VPT, 2>(i));
            const int c = (i * tx + x) * 8;
            if (inside(c)) {
                *reinterpret_cast<uint32_t*>(q + (c >> 1)) = mx4_pack8(y[i], mx4_inv_scale(byte));
            }
        }
    }
}

// --------------------------------------------------------------------------
// Forward, rows of at most 8 * VPT * blockDim.x columns: a row's values stay in
// registers between the sum of squares and the quantisation, so memory is read
// once.  Row blockIdx.x * blockDim.y + threadIdx.y; thread t holds the eights
// t, t + blockDim.x, ... of the row, so that 16 neighbouring lanes hold a group
// of 128.  FULL: the threads cover the rows and columns exactly, nothing is tested.
// --------------------------------------------------------------------------
template <typename T, typename W, int BITS, int VPT, bool FULL>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rmsnorm_quant_kernel(const NormParams p)
{
    const int tx = blockDim.x, x = threadIdx.x;
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool row_ok = FULL || r < p.rows;
    auto inside = [&](int c) { return FULL || (row_ok && c < p.cols); };
    Vec8<T> a[VPT];
    Vec8<W> w0;
    float ss = 0.f;
    grid_begin();
    {
        const T* src = static_cast<const T*>(p.x) + r * p.ldx;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * tx + x) * 8;
            if (!FULL) a[i].zero();
            if (inside(c)) load_stream(a[i], src + c);
        }
    }
    if (p.res != nullptr) {
        const T* res = static_cast<const T*>(p.res) + r * p.ldr;
        T* h = static_cast<T*>(p.h) + r * p.ldh;
        Vec8<T> b[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * tx + x) * 8;
            if (!FULL) b[i].zero();
            if (inside(c)) load_stream(b[i], res + c);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * tx + x) * 8;
            add_round(a[i], b[i]);
            if (inside(c)) store_vec(h + c, a[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) ss = sum_squares(eight_of(a[i]), ss);
    ss = row_sum(ss);
    // the first weights arrive during the reciprocal root, but not fp32 weights of bf16
    // rows, whose registers cost a CTA an SM (16640 x 8192 without residual 85 -> 101 us)
    constexpr bool kEarly = VPT == 1 || sizeof(W) <= sizeof(T);
    auto weights = [&](int c) {
        if (!FULL) w0.zero();
        if (inside(c)) load_kept(w0, static_cast<const W*>(p.w) + c);
    };
    if (kEarly) weights(x * 8);
    const float rstd = rstd_of(ss, p.inv_cols, p.eps);
    if (row_ok && x == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    Eight y[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * tx + x) * 8;
        if (!kEarly || i > 0) weights(c);
        y[i] = normalise(eight_of(a[i]), rstd, eight_of(w0));
    }
    if (p.y != nullptr) {
        T* dst = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (inside((i * tx + x) * 8)) store8(dst + (i * tx + x) * 8, y[i]);
    }
    quantise_store<BITS, VPT, FULL>(p, r, row_ok, tx, x, y);
}

// --------------------------------------------------------------------------
// A ring of row blocks in shared memory: a CTA goes over blocks blockIdx.x,
// + gridDim.x, .. of `ty` rows each, with `slots` blocks of up to three matrices
// in flight (bulk copies, whole rows), so that the next rows arrive while this one
// waits for its sum.  Warp 0 refills a slot once every warp has arrived on its
// empty barrier.  The backward pass uses it, whose CTAs must live long to keep
// their sums of dw; the forward pass is faster with a CTA per row and many of them
// on an SM (16640 x 8192 bf16 with residual: 144-147 us, over a ring 203).
//
// A wait that runs out (bounded as everywhere) raises the error flag and the
// CTA's abort flag and goes on: the row's barriers stay matched and the kernel
// ends, since every later wait returns at once.
// --------------------------------------------------------------------------
constexpr int kRingMats = 3;
constexpr uint64_t kRingWaitNs = 2000000000ull;

struct RowRing {
    const void* src[kRingMats];     // nullptr: none
    int64_t pitch[kRingMats];       // bytes from row to row
    int64_t rows;
    uint32_t row_bytes;
    int tx, ty, slots;              // threads per row, rows per block, ring depth
    int* err;
};

struct RingView {
    uint32_t base, bars;
    uint32_t mat_bytes, slot_bytes;
    int slots;
    volatile int* abort_flag;
    __device__ __forceinline__ uint32_t full(int s) const { return bars + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8u * (slots + s); }
};

// Shared memory of a ring: the slots, then its barriers and the abort flag.
__host__ __device__ constexpr uint32_t ring_smem(uint32_t row_bytes, int ty, int mats, int slots)
{
    return (uint32_t)slots * (uint32_t)mats * (uint32_t)ty * row_bytes + 16u * (uint32_t)slots + 16u;
}

// Block b into slot s (warp 0).
__device__ __forceinline__ void ring_issue(const RowRing& g, const RingView& v, int64_t b, int s)
{
    const int lane = threadIdx.x & 31;
    const int64_t r0 = b * g.ty;
    const int n = (int)min((int64_t)g.ty, g.rows - r0);
    const uint32_t mats = v.slot_bytes / v.mat_bytes;
    if (lane == 0) mbar_arrive_expect_tx(v.full(s), mats * (uint32_t)n * g.row_bytes);
    __syncwarp();
    uint32_t dst = v.base + (uint32_t)s * v.slot_bytes;
#pragma unroll
    for (int m = 0; m < kRingMats; ++m) {
        if (g.src[m] == nullptr) continue;
        const uint8_t* src = static_cast<const uint8_t*>(g.src[m]) + r0 * g.pitch[m];
        if (g.pitch[m] == (int64_t)g.row_bytes) {
            if (lane == 0) bulk_load(dst, src, (uint32_t)n * g.row_bytes, v.full(s));
        } else {
            for (int i = lane; i < n; i += 32)
                bulk_load(dst + (uint32_t)i * g.row_bytes, src + i * g.pitch[m], g.row_bytes, v.full(s));
        }
        dst += v.mat_bytes;
    }
}

// Barriers, and the CTA's first blocks.
__device__ __forceinline__ RingView ring_init(const RowRing& g, uint8_t* smem, int64_t blocks)
{
    const int mats = (g.src[0] != nullptr) + (g.src[1] != nullptr) + (g.src[2] != nullptr);
    RingView v;
    v.base = smem_u32(smem);
    v.mat_bytes = (uint32_t)g.ty * g.row_bytes;
    v.slot_bytes = (uint32_t)mats * v.mat_bytes;
    v.slots = g.slots;
    v.bars = v.base + (uint32_t)g.slots * v.slot_bytes;
    v.abort_flag = reinterpret_cast<volatile int*>(smem + (uint32_t)g.slots * v.slot_bytes + 16u * g.slots);
    if (threadIdx.x == 0) {
        for (int s = 0; s < g.slots; ++s) {
            mbar_init(v.full(s), 1);
            mbar_init(v.empty(s), blockDim.x >> 5);
        }
        *v.abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    grid_begin();
    if (threadIdx.x < 32)
        for (int s = 0; s < g.slots; ++s)
            if (blockIdx.x + (int64_t)s * gridDim.x < blocks) ring_issue(g, v, blockIdx.x + (int64_t)s * gridDim.x, s);
    return v;
}

__device__ __forceinline__ bool ring_wait(const RowRing& g, const RingView& v, uint32_t bar, uint32_t parity)
{
    if (mbar_wait_limit(bar, parity, v.abort_flag, kRingWaitNs)) return true;
    *v.abort_flag = 1;
    atomicOr(g.err, 1);
    return false;
}

// Slot s (in the `phase`-th use) of block b is read: warp 0 refills it.
__device__ __forceinline__ void ring_release(const RowRing& g, const RingView& v, int64_t b, int64_t blocks, int s,
                                             uint32_t phase)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(v.empty(s));
    const int64_t next = b + (int64_t)g.slots * gridDim.x;
    if (threadIdx.x < 32 && next < blocks) {
        const bool ok = ring_wait(g, v, v.empty(s), phase);
        if (__all_sync(0xffffffffu, ok)) ring_issue(g, v, next, s);
    }
}

// Sum over the tx threads of row y of a block (tx = 16, or a multiple of 32; the
// row's warps meet at named barrier 1 + y).  `part`: 16 floats, a multiple of
// four for each row.
__device__ __forceinline__ float ring_row_sum(float v, int tx, int x, int y, float* part)
{
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tx == 16) return v;
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (tx == 32) return v;
    float* mine = part + y * ((tx + 127) >> 7 << 2);
    if ((x & 31) == 0) mine[x >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + y), "r"(tx) : "memory");
    return sum_parts(mine, tx >> 5);
}

// Eight values of the ring's row at byte offset `at`.
template <typename T>
__device__ __forceinline__ Vec8<T> ring_vec(uint32_t at)
{
    Vec8<T> v;
    if constexpr (sizeof(T) == 2) {
        v.raw = lds_u4(at);
    } else {
        v.a = lds128(at);
        v.b = lds128(at + 16);
    }
    return v;
}

// --------------------------------------------------------------------------
// Forward, rows of any width: one CTA per row goes over it twice and takes the
// second look at h from memory (the caches, mostly).
// --------------------------------------------------------------------------
template <typename T, int BITS>
__global__ void __launch_bounds__(512) rmsnorm_quant_wide_kernel(const NormParams p)
{
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* res = static_cast<const T*>(p.res) + r * p.ldr;
    T* h = static_cast<T*>(p.h) + r * p.ldh;
    float ss = 0.f;
    grid_begin();
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.cols; c += (int64_t)blockDim.x * 8) {
        Vec8<T> a;
        load_stream(a, x + c);
        if (p.res != nullptr) {
            Vec8<T> b;
            load_stream(b, res + c);
            add_round(a, b);
            store_vec(h + c, a);
        }
        ss = sum_squares(eight_of(a), ss);
    }
    ss = row_sum(ss);
    const float rstd = rstd_of(ss, p.inv_cols, p.eps);
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[r] = rstd;
    // each thread reads back what it wrote itself; whole warps take part in the
    // groups' maxima
    const T* src = p.res != nullptr ? h : x;
    const int64_t top = (p.cols + 255) / 256 * 256;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < top; c += (int64_t)blockDim.x * 8) {
        Eight y[1] = {eight_zero()};
        if (c < p.cols) {
            Vec8<T> a;
            load_stream(a, src + c);
            y[0] = normalise(eight_of(a), rstd, load_weight8(p.w, p.w_f32, c));
            if (p.y != nullptr) store8(static_cast<T*>(p.y) + r * p.ldy + c, y[0]);
        }
        quantise_store<BITS, 1, false>(p, r, true, 0, (int)(c >> 3), y);
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
    float* dw;                  // dw itself, where one cluster takes all rows
    float* dot;                 // [rows] mean(g n) (wide rows only)
    int64_t rows, cols, lddy, ldh, lddh, lddx;
    int w_f32;
};

// Over a ring of dy, h and dh, rows of at most 8 * VPT * tx columns: a thread
// keeps its columns' sums of dw in registers over all its rows, and its weights
// where they have the rows' type (else they come from L1 with each row, beside
// which the ring leaves little of L1: 16640 x 8192 bf16 took 200 to 245 us so);
// the CTA's rows of sums are added at the end, in order, into row blockIdx.x of
// `part`.  Two CTAs of 256 threads an SM hide each other's sums and barriers: one
// of 512, over two rows at a time, took 247 us where two took 195.
template <typename T, int VPT, int THREADS, bool WREG, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, (VPT == 1 ? 1024 : 512) / THREADS) rmsnorm_back_kernel(const NormBackParams p, const RowRing g)
{
    extern __shared__ __align__(128) uint8_t ring_raw[];
    __shared__ __align__(16) float part[2][16];
    const int64_t blocks = (g.rows + g.ty - 1) / g.ty;
    const RingView v = ring_init(g, ring_raw, blocks);
    const int y = (int)threadIdx.x / g.tx, x = (int)threadIdx.x - y * g.tx;
    Eight dw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) dw[i] = eight_zero();
    Vec8<T> wr[WREG ? VPT : 1];
    if constexpr (WREG) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g.tx + x) * 8;
            wr[i].zero();
            if (c < p.cols) load_stream(wr[i], static_cast<const T*>(p.w) + c);
        }
    }
    auto weight = [&](int i, int c) {
        if constexpr (WREG) return eight_of(wr[i]);
        else return load_weight8(p.w, p.w_f32, c);
    };
    const float inv = 1.f / (float)p.cols;
    int s = 0, flip = 0;
    uint32_t phase = 0;
    // a row's rstd is loaded a block ahead
    const int64_t r_first = (int64_t)blockIdx.x * g.ty + y;
    float rstd_next = r_first < p.rows ? ld_f1(p.rstd + r_first) : 0.f;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, flip ^= 1) {
        const int64_t r = b * g.ty + y;
        const bool row_ok = r < p.rows;
        const float rstd = rstd_next;
        const int64_t r_next = r + (int64_t)gridDim.x * g.ty;
        rstd_next = r_next < p.rows ? ld_f1(p.rstd + r_next) : 0.f;
        ring_wait(g, v, v.full(s), phase);
        const uint32_t at = v.base + (uint32_t)s * v.slot_bytes + (uint32_t)y * g.row_bytes;
        // n = h rstd:  dw += dy n,  dot = sum dy w h
        float2 dot2 = make_float2(0.f, 0.f);
        const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g.tx + x) * 8;
            if (row_ok && c < p.cols) {
                const Eight w = weight(i, c);
                const Eight dy = eight_of(ring_vec<T>(at + (uint32_t)c * sizeof(T)));
                const Eight h = eight_of(ring_vec<T>(at + v.mat_bytes + (uint32_t)c * sizeof(T)));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = fmul2(dy.v[j], h.v[j]);
                    dw[i].v[j] = ffma2(t, rstd2, dw[i].v[j]);
                    dot2 = ffma2(t, w.v[j], dot2);
                }
            }
        }
        // two sets of partial sums: a row's warps may be a block apart
        const float dot = ring_row_sum(dot2.x + dot2.y, g.tx, x, y, part[flip]);
        // dx = rstd (dy w - n mean(g n)) + dh,  mean(g n) = rstd dot / cols (in this order:
        // the cube of rstd may leave fp32's range where none of these does)
        const float k = -(rstd * rstd) * (rstd * (dot * inv));
        const float2 k2 = make_float2(k, k);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * g.tx + x) * 8;
            if (row_ok && c < p.cols) {
                const Eight w = weight(i, c);
                const Eight dy = eight_of(ring_vec<T>(at + (uint32_t)c * sizeof(T)));
                const Eight h = eight_of(ring_vec<T>(at + v.mat_bytes + (uint32_t)c * sizeof(T)));
                Eight f = eight_zero();
                if (p.dh != nullptr) f = eight_of(ring_vec<T>(at + 2 * v.mat_bytes + (uint32_t)c * sizeof(T)));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f.v[j] = ffma2(fmul2(dy.v[j], w.v[j]), rstd2, ffma2(h.v[j], k2, f.v[j]));
                store8(static_cast<T*>(p.dx) + r * p.lddx + c, f);
            }
        }
        ring_release(g, v, b, blocks, s, phase);
        if (++s == g.slots) { s = 0; phase ^= 1u; }
    }
    // the ring is empty: its memory takes the rows of sums
    float* out = p.part + (int64_t)blockIdx.x * p.cols;
    float* sums = reinterpret_cast<float*>(ring_raw);
    const bool direct = !CLUSTER && g.ty == 1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * g.tx + x) * 8;
        if (c < p.cols) store8(direct ? out + c : sums + (int64_t)y * p.cols + c, dw[i]);
    }
    if (direct) return;
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float t = sums[c];
        for (int i = 1; i < g.ty; ++i) t += sums[(int64_t)i * p.cols + c];
        (CLUSTER ? sums : out)[c] = t;
    }
    if constexpr (CLUSTER) {
        // few rows: the cluster's CTAs add each other's sums, in rank order, from shared memory
        __syncthreads();
        cluster_sync_all();
        const uint32_t n = gridDim.x;
        for (int c = (int)(blockIdx.x * blockDim.x + threadIdx.x); c < p.cols; c += (int)(n * blockDim.x)) {
            float t = 0.f;
            for (uint32_t i = 0; i < n; ++i) t += lds_cluster(mapa_shared(v.base + 4u * (uint32_t)c, i));
            p.dw[c] = t;
        }
        __syncthreads();
        cluster_sync_all();
    }
}

// Rows of any width, first launch: dot[r] = mean(g n).
template <typename T>
__global__ void __launch_bounds__(512) rmsnorm_back_dot_kernel(const NormBackParams p)
{
    const int64_t r = blockIdx.x;
    float2 dot2 = make_float2(0.f, 0.f);
    grid_begin();
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.cols; c += (int64_t)blockDim.x * 8) {
        Vec8<T> a, b;
        load_stream(a, static_cast<const T*>(p.dy) + r * p.lddy + c);
        load_stream(b, static_cast<const T*>(p.h) + r * p.ldh + c);
        const Eight dy = eight_of(a), h = eight_of(b), w = load_weight8(p.w, p.w_f32, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) dot2 = ffma2(fmul2(dy.v[j], h.v[j]), w.v[j], dot2);
    }
    float dot = dot2.x + dot2.y;
    dot = row_sum(dot) * p.rstd[r];
    if (threadIdx.x == 0) p.dot[r] = dot / (float)p.cols;
}

// Second launch: CTA (x, y) goes over rows y, y + gridDim.y, ... of its 2048
// columns.
template <typename T>
__global__ void __launch_bounds__(256) rmsnorm_back_wide_kernel(const NormBackParams p)
{
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    grid_begin();
    if (c >= p.cols) return;
    const Eight w = load_weight8(p.w, p.w_f32, c);
    Eight dw = eight_zero();
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const float rstd = p.rstd[r], k = -(rstd * rstd) * p.dot[r];
        const float2 rstd2 = make_float2(rstd, rstd), k2 = make_float2(k, k);
        Vec8<T> a, b, d;
        load_stream(a, static_cast<const T*>(p.dy) + r * p.lddy + c);
        load_stream(b, static_cast<const T*>(p.h) + r * p.ldh + c);
        d.zero();
        if (p.dh != nullptr) load_stream(d, static_cast<const T*>(p.dh) + r * p.lddh + c);
        const Eight dy = eight_of(a), h = eight_of(b);
        Eight f = eight_of(d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dw.v[j] = ffma2(fmul2(dy.v[j], h.v[j]), rstd2, dw.v[j]);
            f.v[j] = ffma2(fmul2(dy.v[j], w.v[j]), rstd2, ffma2(h.v[j], k2, f.v[j]));
        }
        store8(static_cast<T*>(p.dx) + r * p.lddx + c, f);
    }
    store8(p.part + (int64_t)blockIdx.y * p.cols + c, dw);
}

// dw[c] = sum over the parts, 32 columns a CTA: warp w adds parts w, w + 32, ..,
// ten loads in flight (the usual two parts an SM in one round trip to L2), and the
// warps' sums are added in a tree.
constexpr int kDwWarps = 32;

__global__ void __launch_bounds__(32 * kDwWarps) rmsnorm_dw_kernel(const float* part, int parts, int64_t cols,
                                                                   float* dw)
{
    __shared__ float s[kDwWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    grid_begin();
    float sum = 0.f;
    if (c < cols) {
        for (int i = warp; i < parts; i += 10 * kDwWarps) {
            float v[10];
#pragma unroll
            for (int j = 0; j < 10; ++j)
                v[j] = i + kDwWarps * j < parts ? ld_l2_f1(part + (int64_t)(i + kDwWarps * j) * cols + c) : 0.f;
#pragma unroll
            for (int j = 0; j < 10; ++j) sum += v[j];
        }
    }
    s[warp][lane] = sum;
    __syncthreads();
    // warp w adds column w's sums: lane l holds warp l's
    float t = s[lane][warp];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int64_t col = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && col < cols) dw[col] = t;
}

}  // namespace fp8bs
