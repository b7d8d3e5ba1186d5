// gemm_fp4_kernel.cuh -- product of two microscaled 4-bit matrices on single CTAs
// (tcgen05 kind::mxf4.block_scale): few tokens, or an output of few tiles.
//
//   D[m,n] = sum_g rA(m,g) rB(n,g) sum_{k in group g} a[m,k] b[n,k],   groups of 32 K.
//
// The tensor cores multiply each product by its two power-of-two factors and
// accumulate in fp32 in TMEM.
//
// B^T's rows (a layer's weight) are the MMA's 128 rows and A's rows (the tokens)
// its BN columns, so that a few tokens need a few accumulator columns only: the
// weight streams through at 128 rows a tile whatever M is, and the number of
// tokens sets BN (16 .. 128).  D^T's columns are D's rows, so a warp stores 32
// consecutive elements of a row of D.
//
// The kernel of few tokens is bound by the weight's bytes and its own latency (one
// token by 5120 x 8192: 5.6 us, of which 3.4 are the bytes at the measured copy
// rate; about 800 cycles of set-up, 800 to the first bytes, 500 a step of 20 KB,
// 1300 from the last step to the accumulator, 900 for the sums).
//
// One unit per CTA: a tile and a part of K.  Two CTAs share an SM, so that one's
// set-up and epilogue run under the other's loads.  A tile's K is split over the
// CTAs of a cluster (1, 2, 4 or 8): every group of four columns has an owner, the
// others send it their sums (st.async into its shared memory, counted on its
// mbarrier), and the owner adds them in rank order.  That needs no second launch,
// no workspace and no barrier after the loads (two cluster barriers and reads of
// the peers' memory cost 2 us of 7.5 at one token by 5120 x 8192).  Very long K is
// split further, over clusters, through a workspace and splitk_reduce_kernel.
//
// Warps:
//   warp 0      producer: per step of 256 K (128 bytes a row) one TMA tile of B^T
//               (128 rows) and of A (BN rows), 128-byte swizzle, and their scale
//               tiles (two 512-byte tiles, adjacent in memory) by bulk copies, into
//               a ring.
//   warp 1      TMEM allocation; lane 0 issues the step's MMAs (K = 64 each, only
//               those that start below K).
//   warps 2-5   one per TMEM lane quarter: write each step's scale factors to TMEM
//               (tcgen05.st; copies by tcgen05.cp queue with the MMAs, about 85
//               cycles each), then the epilogue.
// A stage's scale columns in TMEM are written again only after the MMAs that read
// them have completed, since the producer refills a stage after its commit.
// Scale bytes of rows past the matrices' last are not set by anyone: they reach
// only accumulator rows and columns that are not stored.
//
// Every mbarrier wait is bounded as in gemm_bs_kernel.cuh.  A CTA that gives up
// sends nothing; the owners wait for a peer's sums three times as long as a
// peer's own waits can last, so that nothing is sent to a CTA that has left.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "ptx_bs.cuh"
#include "ptx_fp4.cuh"
#include "mx4.cuh"
#include "quant_kernels.cuh"
#include "gemm_kernel.cuh"

namespace fp8bs {

constexpr int kF4Rows = 128;                   // rows of B^T per tile
constexpr int kF4StepK = 256;                  // K per step: 128 bytes
constexpr int kF4MmaK = 64;
constexpr int kF4MaxCluster = 8;               // CTAs that share a tile's K
constexpr int kF4Threads = 32 * 6;
constexpr uint32_t kF4Prefetch = 4;            // steps of the weight that are sent for early
constexpr uint32_t kQuadBytes = kF4Rows * 16;  // four columns of a tile's 128 rows, fp32

struct Fp4Params {
    int32_t M, N, K;
    int32_t steps;              // ceil(K / K per step)
    int32_t kcs;                // scale tiles per 128 rows: ceil(K / 128)
    int32_t tiles_m, tiles_n;
    int32_t splits;             // parts of K that go through the workspace
    int32_t band;               // weight tiles per band of the tile order
    int64_t num_units;          // tiles_m * tiles_n * splits
    const uint8_t* B;           // B^T (the tensor maps' too) and its leading dimension
    int64_t ldb;
    const uint8_t* sfa;         // scale tiles of A (tokens) and of B^T
    const uint8_t* sfb;
    void* D;
    int64_t ldd;
    int32_t out_f32;
    float* ws;                  // partial sums [splits][M][ldw] fp32
    int64_t ldw;
    int* err;
};

template <int BN>
struct Fp4Cfg {
    static constexpr uint32_t w_bytes = kF4Rows * 128;      // 16 KB
    static constexpr uint32_t t_bytes = BN * 128;
    static constexpr uint32_t sf_bytes = 2 * 2 * kSfTileBytes;   // B^T's block and A's, two tiles each
    // sums received: [rank][owned group of four columns][128 rows][4] fp32, in
    // memory of their own, or for the widest tile in the stages' place (then the
    // cluster meets once more, when all its products are done)
    static constexpr uint32_t red_bytes = (BN < 32 ? 32 : BN) * kF4Rows * 4;
    static constexpr bool red_own = BN <= 64;
    // two CTAs per SM: at most 113 KB of shared memory and 256 columns of TMEM each
    static constexpr int stages = BN <= 32 ? 4 : 3;
    static constexpr uint32_t acc_cols = BN < 32 ? 32 : BN;
    static constexpr uint32_t sf_cols = 16;                 // two chunks x (B^T's 4 words, A's 4)
    static constexpr uint32_t tmem_cols = 256;
    static_assert(acc_cols + stages * sf_cols <= tmem_cols, "scale factors exceed TMEM");
    // shared memory
    static constexpr uint32_t t_off = stages * w_bytes;
    static constexpr uint32_t sf_off = t_off + stages * t_bytes;
    static constexpr uint32_t red_off = red_own ? sf_off + stages * sf_bytes : 0;
    static constexpr uint32_t bar_off = sf_off + stages * sf_bytes + (red_own ? red_bytes : 0);
    static_assert(red_own || red_bytes <= sf_off, "sums received exceed the stages");
    static constexpr uint32_t n_bars = 3 * stages + 2;
    static constexpr uint32_t misc_off = bar_off + n_bars * 8;
    static constexpr uint32_t alloc = misc_off + 16 + 1024;
    static_assert(2 * (alloc + 1024) <= 233472, "shared memory of two CTAs per SM");
    static_assert(t_off % 1024 == 0 && t_bytes % 1024 == 0, "swizzled tiles 1024-byte aligned");
};

// Unit u: bands of p.band weight tiles, all token tiles of a band before the next
// band, so that concurrent CTAs share both operands in L2.
__device__ __forceinline__ void fp4_unit(const Fp4Params& p, uint32_t u, int& tm, int& tn, int& split)
{
    uint32_t tile = u;
    split = 0;
    if (p.splits > 1) {
        tile = u / (uint32_t)p.splits;
        split = (int)(u - tile * (uint32_t)p.splits);
    }
    if (p.tiles_m == 1) {
        tm = 0;
        tn = (int)tile;
        return;
    }
    const uint32_t per_band = (uint32_t)(p.band * p.tiles_m);
    const uint32_t band = tile / per_band;
    const uint32_t in = tile - band * per_band;
    const int n0 = (int)band * p.band;
    const uint32_t width = (uint32_t)min(p.band, p.tiles_n - n0);
    tm = (int)(in / width);
    tn = n0 + (int)(in - (uint32_t)tm * width);
}

// `cnt` (at most CNT) consecutive columns of D^T, i.e. one element in each of
// that many rows of D, ld elements apart.
template <int CNT>
__device__ __forceinline__ void fp4_store(float* dst, int64_t ld, const float (&v)[CNT], int cnt)
{
    if (cnt >= CNT) {
#pragma unroll
        for (int c = 0; c < CNT; ++c, dst += ld) *dst = v[c];
    } else {
#pragma unroll
        for (int c = 0; c < CNT; ++c, dst += ld)
            if (c < cnt) *dst = v[c];
    }
}
template <int CNT>
__device__ __forceinline__ void fp4_store(__nv_bfloat16* dst, int64_t ld, const float (&v)[CNT], int cnt)
{
    if (cnt >= CNT) {
#pragma unroll
        for (int c = 0; c < CNT; ++c, dst += ld) *dst = __float2bfloat16_rn(v[c]);
    } else {
#pragma unroll
        for (int c = 0; c < CNT; ++c, dst += ld)
            if (c < cnt) *dst = __float2bfloat16_rn(v[c]);
    }
}

// A tile's accumulator (or, with K split over a cluster, this CTA's quads of it)
// to D or to the workspace.  `dst`: row m0, the lane's column.
template <int BN, typename T>
__device__ __forceinline__ void fp4_store_tile(uint32_t taddr, T* dst, int64_t ld, int cols, bool store)
{
    constexpr int kChunk = BN < 32 ? 16 : 32;
#pragma unroll 1
    for (int c0 = 0; c0 < cols; c0 += kChunk) {
        uint32_t r[kChunk / 16][16];
#pragma unroll
        for (int i = 0; i < kChunk / 16; ++i) tmem_ld_32x32b_x16(taddr + (uint32_t)(c0 + 16 * i), r[i]);
        tmem_ld_wait(r[0]);
#pragma unroll
        for (int i = 1; i < kChunk / 16; ++i) reg_after_wait(r[i]);
        if (store) {
            float v[kChunk];
#pragma unroll
            for (int c = 0; c < kChunk; ++c) v[c] = __uint_as_float(r[c >> 4][c & 15]);
            fp4_store(dst + (int64_t)c0 * ld, ld, v, cols - c0);
        }
    }
}
template <typename T>
__device__ __forceinline__ void fp4_store_quads(uint32_t mine, uint32_t share, uint32_t parts, uint32_t rank,
                                                uint32_t owned, T* dst, int64_t ld, int cols)
{
#pragma unroll 2
    for (uint32_t g = 0; g < owned; ++g) {
        float4 v[kF4MaxCluster];
#pragma unroll
        for (int j = 0; j < kF4MaxCluster; ++j)
            if (j < (int)parts) v[j] = lds128(mine + (uint32_t)j * share + g * kQuadBytes);
        float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int j = 1; j < kF4MaxCluster; ++j)
            if (j < (int)parts) { sum[0] += v[j].x; sum[1] += v[j].y; sum[2] += v[j].z; sum[3] += v[j].w; }
        const int c = (int)(g * parts + rank) * 4;
        fp4_store(dst + (int64_t)c * ld, ld, sum, cols - c);
    }
}

template <int BN>
__global__ void __launch_bounds__(kF4Threads, 2)
gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT, const Fp4Params p)
{
    using C = Fp4Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + C::bar_off;
    auto ab_full = [&](int s) { return bars + 8u * s; };       // operands landed and scale columns written
    auto ab_empty = [&](int s) { return bars + 8u * (C::stages + s); };
    auto sl_full = [&](int s) { return bars + 8u * (2 * C::stages + s); };   // scale tiles landed
    const uint32_t tm_full = bars + 8u * (3 * C::stages);
    const uint32_t red_full = tm_full + 8u;                    // the peers' sums have arrived
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::misc_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), parts = cluster_nctarank();

    int tm, tn, split;
    const int log_parts = 31 - __clz((int)parts);
    fp4_unit(p, blockIdx.x >> log_parts, tm, tn, split);
    const int m0 = tm * BN, n0 = tn * kF4Rows;
    const int cols = min(BN, p.M - m0);                 // columns (tokens) that D has
    const uint32_t quads = (uint32_t)(cols + 3) >> 2;
    // of which this CTA owns quads rank, rank + parts, ..
    const uint32_t owned = quads > rank ? (quads - rank + parts - 1) >> log_parts : 0;

    // this CTA's steps: part of p.splits * parts (steps <= 2^23 and at most 256
    // parts: 32 bits hold the products)
    uint32_t s0 = (uint32_t)p.steps * ((uint32_t)split * parts + rank) >> log_parts;
    uint32_t s1 = (uint32_t)p.steps * ((uint32_t)split * parts + rank + 1) >> log_parts;
    if (p.splits > 1) {
        s0 /= (uint32_t)p.splits;
        s1 /= (uint32_t)p.splits;
    }
    if (p.tiles_m == 1 && warp >= 2) {
        // few tokens: the weight's first steps set out for L2 under the previous kernel.
        // With a norm in front and the weight in memory, 24 x 8192 x 5120 takes 9.5 us
        // for both, without this 10.2; more steps gain no more and cost 0.3 where the
        // weight is in L2 already.
        const int row = n0 + (int)threadIdx.x - 64;
        const uint8_t* w = p.B + (int64_t)row * p.ldb;
        if (row < p.N)
            for (uint32_t st = s0; st < min(s1, s0 + kF4Prefetch); ++st) prefetch_l2(w + (int64_t)st * 128);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::stages; ++s) {
            mbar_init(ab_full(s), 1 + 4);
            mbar_init(ab_empty(s), 1);
            mbar_init(sl_full(s), 1);
        }
        mbar_init(tm_full, 1);
        mbar_init(red_full, 1);
        *abort_flag = 0;
        fence_barrier_init();
        if (parts > 1) mbar_arrive_expect_tx(red_full, (parts - 1) * owned * kQuadBytes);
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmT);
    }
    if (warp == 1) {
        tmem_alloc(sbase + C::misc_off, C::tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the peers may send once every CTA of the cluster has passed here
    if (parts > 1) cluster_arrive();
    const uint32_t tmem_base = *tmem_slot;
    // everything above may run under the previous kernel's tail; the next one's
    // may run under this
    grid_begin();

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.err, 1);
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            uint32_t filled = 0, fill_par = 0;
            for (int st = (int)s0; st < (int)s1; ++st) {
                if (!mbar_wait_limit(ab_empty(stage), phase ^ 1u, abort_flag, kWaitLimitNs)) { ok = false; break; }
                const uint32_t bytes = kSfTileBytes * (uint32_t)min(2, p.kcs - 2 * st);
                mbar_arrive_expect_tx(sl_full(stage), 2 * bytes);
                const uint32_t sf = sbase + C::sf_off + stage * C::sf_bytes;
                bulk_load(sf, p.sfb + ((int64_t)tn * p.kcs + 2 * st) * kSfTileBytes, bytes, sl_full(stage));
                bulk_load(sf + 2 * kSfTileBytes, p.sfa + ((int64_t)(m0 >> 7) * p.kcs + 2 * st) * kSfTileBytes, bytes,
                          sl_full(stage));
                mbar_arrive_expect_tx(ab_full(stage), C::w_bytes + C::t_bytes);
                tma_load_2d(sbase + stage * C::w_bytes, &tmW, ab_full(stage), st * 128, n0);
                tma_load_2d(sbase + C::t_off + stage * C::t_bytes, &tmT, ab_full(stage), st * 128, m0);
                filled |= 1u << stage;
                fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
                if (++stage == C::stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) give_up();
            // every issued load lands before the CTA exits or its shared memory is used again
            for (int s = 0; s < C::stages; ++s)
                if (filled >> s & 1u) {
                    mbar_wait_bounded(sl_full(s), fill_par >> s & 1u, nullptr, kDrainLimitNs);
                    mbar_wait_bounded(ab_full(s), fill_par >> s & 1u, nullptr, kDrainLimitNs);
                }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int st = (int)s0; st < (int)s1; ++st) {
                if (!mbar_wait_limit(ab_full(stage), phase, abort_flag, kWaitLimitNs)) { ok = false; break; }
                tc_fence_after();
                const uint32_t sf = tmem_base + C::acc_cols + (uint32_t)stage * C::sf_cols;
                const uint64_t wd = smem_desc_k_sw128(sbase + stage * C::w_bytes);
                const uint64_t td = smem_desc_k_sw128(sbase + C::t_off + stage * C::t_bytes);
                const int left = p.K - st * kF4StepK;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t id = (uint32_t)(k & 1) * 2u;
                    const uint32_t col = (sf + (uint32_t)(k >> 1) * (C::sf_cols / 2)) | (id << 30);
                    if (k * kF4MmaK < left)
                        umma_f4_bs(tmem_base, wd + 2 * k, td + 2 * k, idesc_e2m1_bs(kF4Rows, BN, id), col, col + 4,
                                   (st > (int)s0 || k > 0) ? 1u : 0u);
                }
                umma_commit(ab_empty(stage));
                if (++stage == C::stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) give_up();
            // also when nothing was issued: the epilogue and the end of the CTA wait for it
            umma_commit(tm_full);
            mbar_wait_bounded(tm_full, 0, nullptr, kDrainLimitNs);
        }
    } else {
        // ---------------------------------------------------------------- scale-factor writers
        const int lq = warp & 3;
        const uint32_t lane_addr = tmem_base + ((uint32_t)(lq * 32) << 16);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int st = (int)s0; st < (int)s1; ++st) {
            if (!mbar_wait_limit(sl_full(stage), phase, abort_flag, kWaitLimitNs)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // lane l: row l of each tile (its four words are rows l, l + 32, ..); chunk c of the
            // step: B^T's block, A's block
            const uint32_t src = sbase + C::sf_off + stage * C::sf_bytes + (uint32_t)lane * 16u;
            uint32_t r[16];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 v = lds_u4(src + (2 * j + c) * kSfTileBytes);
                    r[8 * c + 4 * j] = v.x;
                    r[8 * c + 4 * j + 1] = v.y;
                    r[8 * c + 4 * j + 2] = v.z;
                    r[8 * c + 4 * j + 3] = v.w;
                }
            if (BN == 64 && (m0 & 64)) {
                // the tile's rows of A are the second half of their 128-row block
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    r[8 * c + 4] = r[8 * c + 6];
                    r[8 * c + 5] = r[8 * c + 7];
                }
            }
            tmem_st_32x32b_x16(lane_addr + C::acc_cols + (uint32_t)stage * C::sf_cols, r);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ab_full(stage));
            if (++stage == C::stages) { stage = 0; phase ^= 1u; }
        }
        // ---------------------------------------------------------------- epilogue
        if (ok && !mbar_wait_limit(tm_full, 0, abort_flag, kWaitLimitNs)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) give_up();
        tc_fence_after();
        const int row = lq * 32 + lane, n = n0 + row;
        const bool bf16 = p.splits == 1 && !p.out_f32;
        const int64_t ld = p.splits > 1 ? p.ldw : p.ldd;
        float* dst32 = p.splits > 1 ? p.ws + ((int64_t)split * p.M + m0) * ld + n
                                    : static_cast<float*>(p.D) + (int64_t)m0 * ld + n;
        __nv_bfloat16* dst16 = static_cast<__nv_bfloat16*>(p.D) + (int64_t)m0 * ld + n;
        if (parts > 1) {
            cluster_wait();
            if (!C::red_own) {
                cluster_arrive();
                cluster_wait();
            }
            // slot of (rank, owned quad i): 128 rows of 16 bytes
            const uint32_t mine = sbase + C::red_off + (uint32_t)row * 16u;
            const uint32_t share = ((quads + parts - 1) >> log_parts) * kQuadBytes;
            if (ok) {
                uint32_t owner = 0, i = 0;
#pragma unroll 1
                for (uint32_t q0 = 0; q0 < quads; q0 += 4) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(lane_addr + q0 * 4, r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (q0 + j < quads) {
                            const uint32_t at = mine + rank * share + i * kQuadBytes;
                            if (owner == rank) sts128(at, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                            else st_async_v4(mapa_shared(at, owner), r + 4 * j, mapa_shared(red_full, owner));
                            if (++owner == parts) { owner = 0; ++i; }
                        }
                    }
                }
            }
            // a thread reads back the rows that it (and its like in the peers) wrote; a CTA that
            // gave up stays as well until what its peers send it has arrived
            if (owned > 0 && !mbar_wait_limit(red_full, 0, nullptr, 3 * kWaitLimitNs)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (ok && n < p.N) {
                if (bf16) fp4_store_quads(mine, share, parts, rank, owned, dst16, ld, cols);
                else fp4_store_quads(mine, share, parts, rank, owned, dst32, ld, cols);
            }
        } else if (ok) {
            if (bf16) fp4_store_tile<BN>(lane_addr, dst16, ld, cols, n < p.N);
            else fp4_store_tile<BN>(lane_addr, dst32, ld, cols, n < p.N);
        }
        if (!ok && lane == 0) give_up();
    }
    if (parts > 1 && warp < 2) {
        __syncwarp();
        cluster_wait();
        if (!C::red_own) {
            cluster_arrive();
            cluster_wait();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::tmem_cols);
}

}  // namespace fp8bs
