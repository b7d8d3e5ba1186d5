// gemm_fp4_kernel.cuh -- product of two microscaled 4-bit matrices on single CTAs
// (tcgen05 kind::mxf4.block_scale):
//
//   D[m,n] = sum_g rA(m,g) rB(n,g) sum_{k in group g} a[m,k] b[n,k],   groups of 32 K.
//
// The tensor cores multiply each product by its two power-of-two factors and
// accumulate a unit's whole K range in fp32 in TMEM.
//
// B^T's rows (a layer's weight) are the MMA's 128 rows and A's rows (the tokens)
// its BN columns, so that a few tokens need a few accumulator columns only: the
// weight streams through at 128 rows a tile whatever M is, and the number of
// tokens sets BN (16 .. 256).  D^T's columns are D's rows, so a warp stores 32
// consecutive elements of a row of D.
//
// One persistent CTA per SM, 4 + kEpiWarps warps:
//   warp 0      producer: per step of 256 K (128 bytes a row) one TMA tile of B^T
//               (128 rows) and of A (BN rows), 128-byte swizzle, and their scale
//               tiles (two 512-byte tiles per 128 rows, adjacent in memory) by
//               bulk copies, into a ring of kStages.
//   warp 1      TMEM allocation; lane 0 copies a stage's scale tiles into that
//               stage's TMEM columns (tcgen05.cp) and issues the step's MMAs (K =
//               64 each, only those that start below K).
//   warps 4..   epilogue: TMEM -> registers, release the accumulator, convert and
//               store.
// A stage's scale columns in TMEM are written again only after the MMAs that read
// them have completed, since the producer refills a stage after its commit.
// Scale bytes of rows past the matrices' last are not set by anyone: they reach
// only accumulator rows and columns that are not stored.
//
// Every mbarrier wait is bounded as in gemm_bs_kernel.cuh.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "ptx_bs.cuh"
#include "ptx_fp4.cuh"
#include "mx4.cuh"
#include "gemm_kernel.cuh"

namespace fp8bs {

constexpr int kF4Rows = 128;                   // rows of B^T per tile
constexpr int kF4StepK = 256;                  // K per step: 128 bytes
constexpr int kF4MmaK = 64;

struct Fp4Params {
    int32_t M, N, K;
    int32_t steps;              // ceil(K / 256)
    int32_t kcs;                // scale tiles per 128 rows: ceil(K / 128)
    int32_t tiles_m, tiles_n;
    int32_t splits;
    int32_t band;               // weight tiles per band of the tile order
    int64_t num_units;          // tiles_m * tiles_n * splits
    const uint8_t* sfa;         // scale tiles of A (tokens) and of B^T
    const uint8_t* sfb;
    void* D;
    int64_t ldd;
    int32_t out_f32;
    float* ws;                  // split-K partials [splits][M][ldw] fp32
    int64_t ldw;
    int* err;
};

template <int BN>
struct Fp4Cfg {
    static constexpr int sfn = (BN + 127) / 128;            // 128-row blocks of A's scale tiles
    static constexpr int accs = BN <= 128 ? 2 : 1;          // accumulators
    static constexpr int epi_warps = BN <= 64 ? 4 : 8;
    static constexpr int threads = 32 * (4 + epi_warps);
    static constexpr int cols = BN * 4 / epi_warps;         // accumulator columns per epilogue thread
    static constexpr uint32_t w_bytes = kF4Rows * 128;      // 16 KB
    static constexpr uint32_t t_bytes = BN * 128;
    static constexpr uint32_t sf_bytes = (1 + sfn) * 2 * kSfTileBytes;
    static constexpr uint32_t sf_cols = 2 * 4 * (1 + sfn);  // TMEM columns of a stage's factors
    static constexpr int fit = (int)((232448 - 2048) / (w_bytes + t_bytes + sf_bytes));
    static constexpr int stages = fit > 8 ? 8 : fit;
    static constexpr uint32_t sf_col0 = accs * (BN < 32 ? 32 : BN);
    static constexpr uint32_t acc_cols = BN < 32 ? 32 : BN;
    static_assert(sf_col0 + stages * sf_cols <= kTmemCols, "scale factors exceed TMEM");
    // shared memory
    static constexpr uint32_t t_off = stages * w_bytes;
    static constexpr uint32_t sf_off = t_off + stages * t_bytes;
    static constexpr uint32_t bar_off = sf_off + stages * sf_bytes;
    static constexpr uint32_t n_bars = 2 * stages + 2 * accs + 1;
    static constexpr uint32_t misc_off = bar_off + n_bars * 8;
    static constexpr uint32_t alloc = misc_off + 16 + 1024;
    static_assert(alloc <= 232448, "shared memory per CTA");
    static_assert(t_off % 1024 == 0 && t_bytes % 1024 == 0, "swizzled tiles 1024-byte aligned");
};

// Unit u: bands of p.band weight tiles, all token tiles of a band before the next
// band, so that concurrent CTAs share both operands in L2.
__device__ __forceinline__ void fp4_unit(const Fp4Params& p, int64_t u, int& tm, int& tn, int& s0, int& s1, int& split)
{
    const int64_t tile = u / p.splits;
    split = (int)(u - tile * p.splits);
    const int64_t per_band = (int64_t)p.band * p.tiles_m;
    const int64_t band = tile / per_band;
    const int64_t in = tile - band * per_band;
    const int n0 = (int)band * p.band;
    const int width = min(p.band, p.tiles_n - n0);
    tn = n0 + (int)(in % width);
    tm = (int)(in / width);
    s0 = (int)(((int64_t)p.steps * split) / p.splits);
    s1 = (int)(((int64_t)p.steps * (split + 1)) / p.splits);
}

template <int BN>
__global__ void __launch_bounds__(Fp4Cfg<BN>::threads, 1)
gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT, const Fp4Params p)
{
    using C = Fp4Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + C::bar_off;
    auto ab_full = [&](int s) { return bars + 8u * s; };
    auto ab_empty = [&](int s) { return bars + 8u * (C::stages + s); };
    auto tm_full = [&](int a) { return bars + 8u * (2 * C::stages + a); };
    auto tm_empty = [&](int a) { return bars + 8u * (2 * C::stages + C::accs + a); };
    const uint32_t drain_bar = bars + 8u * (2 * C::stages + 2 * C::accs);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::misc_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc_off + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::stages; ++s) {
            mbar_init(ab_full(s), 1);
            mbar_init(ab_empty(s), 1);
        }
        for (int a = 0; a < C::accs; ++a) {
            mbar_init(tm_full(a), 1);
            mbar_init(tm_empty(a), C::epi_warps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmT);
    }
    if (warp == 1) {
        tmem_alloc(sbase + C::misc_off, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

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
            for (int64_t u = blockIdx.x; u < p.num_units && ok; u += gridDim.x) {
                int tm, tn, s0, s1, split;
                fp4_unit(p, u, tm, tn, s0, s1, split);
                const int m0 = tm * BN, n0 = tn * kF4Rows;
                // 128-row blocks of A's scale tiles this tile needs and A has
                const int mb = min(C::sfn, (p.M - m0 + 127) >> 7);
                for (int st = s0; st < s1; ++st) {
                    if (!mbar_wait_bounded(ab_empty(stage), phase ^ 1u, abort_flag, kWaitLimitNs)) { ok = false; break; }
                    const uint32_t bytes = kSfTileBytes * (uint32_t)min(2, p.kcs - 2 * st);
                    mbar_arrive_expect_tx(ab_full(stage), C::w_bytes + C::t_bytes + (1u + mb) * bytes);
                    tma_load_2d(sbase + stage * C::w_bytes, &tmW, ab_full(stage), st * 128, n0);
                    tma_load_2d(sbase + C::t_off + stage * C::t_bytes, &tmT, ab_full(stage), st * 128, m0);
                    const uint32_t sf = sbase + C::sf_off + stage * C::sf_bytes;
                    bulk_load(sf, p.sfb + ((int64_t)tn * p.kcs + 2 * st) * kSfTileBytes, bytes, ab_full(stage));
                    for (int j = 0; j < mb; ++j)
                        bulk_load(sf + (1 + j) * 2 * kSfTileBytes,
                                  p.sfa + ((int64_t)((m0 >> 7) + j) * p.kcs + 2 * st) * kSfTileBytes, bytes,
                                  ab_full(stage));
                    filled |= 1u << stage;
                    fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == C::stages) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) give_up();
            for (int s = 0; s < C::stages; ++s)
                if (filled >> s & 1u) mbar_wait_bounded(ab_full(s), fill_par >> s & 1u, nullptr, kDrainLimitNs);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, issued = false;
            for (int64_t u = blockIdx.x; u < p.num_units && ok; u += gridDim.x) {
                int tm, tn, s0, s1, split;
                fp4_unit(p, u, tm, tn, s0, s1, split);
                const uint32_t d_tmem = tmem_base + (uint32_t)acc * C::acc_cols;
                if (!mbar_wait_bounded(tm_empty(acc), tphase ^ 1u, abort_flag, kWaitLimitNs)) { ok = false; break; }
                for (int st = s0; st < s1; ++st) {
                    if (!mbar_wait_bounded(ab_full(stage), phase, abort_flag, kWaitLimitNs)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t src = sbase + C::sf_off + stage * C::sf_bytes;
                    const uint32_t sf = tmem_base + C::sf_col0 + (uint32_t)stage * C::sf_cols;
                    const int mmas = min(4, (p.K - st * kF4StepK + kF4MmaK - 1) / kF4MmaK);
                    // chunk c of the step: B^T's four columns, then four for each block of A
                    for (int c = 0; c < (mmas + 1) >> 1; ++c)
#pragma unroll
                        for (int j = 0; j <= C::sfn; ++j)
                            tmem_cp_32x128b_x4(sf + c * (C::sf_cols / 2) + 4 * j,
                                               smem_desc_cp_rows16(src + (2 * j + c) * kSfTileBytes));
                    const uint32_t w_addr = sbase + stage * C::w_bytes;
                    const uint32_t t_addr = sbase + C::t_off + stage * C::t_bytes;
                    for (int k = 0; k < mmas; ++k) {
                        const uint32_t id = (uint32_t)(k & 1) * 2u;
                        const uint32_t col = (sf + (uint32_t)(k >> 1) * (C::sf_cols / 2)) | (id << 30);
                        umma_f4_bs(d_tmem, smem_desc_k_sw128(w_addr + k * 32), smem_desc_k_sw128(t_addr + k * 32),
                                   idesc_e2m1_bs(kF4Rows, BN, id), col, col + 4, (st > s0 || k > 0) ? 1u : 0u);
                    }
                    issued = true;
                    if (st + 1 == s1) umma_commit(tm_full(acc));
                    umma_commit(ab_empty(stage));
                    if (++stage == C::stages) { stage = 0; phase ^= 1u; }
                }
                if (++acc == C::accs) { acc = 0; tphase ^= 1u; }
            }
            if (!ok) give_up();
            if (issued) {
                umma_commit(drain_bar);
                mbar_wait_bounded(drain_bar, 0, nullptr, kDrainLimitNs);
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue
        const int lq = warp & 3;
        const int col0 = ((warp - 4) >> 2) * C::cols;
        uint32_t tphase = 0;
        int acc = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < p.num_units; u += gridDim.x) {
            int tm, tn, s0, s1, split;
            fp4_unit(p, u, tm, tn, s0, s1, split);
            if (!mbar_wait_bounded(tm_full(acc), tphase, abort_flag, kWaitLimitNs)) ok = false;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(lq * 32) << 16) + (uint32_t)acc * C::acc_cols + (uint32_t)col0;
            uint32_t r[C::cols / 16][16];
#pragma unroll
            for (int i = 0; i < C::cols / 16; ++i) tmem_ld_32x32b_x16(taddr + 16 * i, r[i]);
            tmem_ld_wait(r[0]);
#pragma unroll
            for (int i = 1; i < C::cols / 16; ++i) reg_after_wait(r[i]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tm_empty(acc));
            if (++acc == C::accs) { acc = 0; tphase ^= 1u; }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;

            const int n = tn * kF4Rows + lq * 32 + lane;
            const int m0 = tm * BN + col0;
            if (n < p.N) {
                if (p.splits > 1 || p.out_f32) {
                    float* dst = p.splits > 1 ? p.ws + ((int64_t)split * p.M + m0) * p.ldw + n
                                              : static_cast<float*>(p.D) + (int64_t)m0 * p.ldd + n;
                    const int64_t ld = p.splits > 1 ? p.ldw : p.ldd;
#pragma unroll
                    for (int c = 0; c < C::cols; ++c)
                        if (m0 + c < p.M) dst[c * ld] = __uint_as_float(r[c >> 4][c & 15]);
                } else {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.D) + (int64_t)m0 * p.ldd + n;
#pragma unroll
                    for (int c = 0; c < C::cols; ++c)
                        if (m0 + c < p.M) dst[c * p.ldd] = __float2bfloat16_rn(__uint_as_float(r[c >> 4][c & 15]));
                }
            }
        }
        if (!ok && lane == 0) give_up();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
}

}  // namespace fp8bs
