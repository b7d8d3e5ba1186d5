// gemm_fp4_pair_kernel.cuh -- product of two microscaled 4-bit matrices on CTA
// pairs (tcgen05 cta_group::2, kind::mxf4.block_scale): the large products.
//
// Same result as gemm_fp4_kernel.cuh, in 256 x 256 tiles: 256 rows of B^T (128
// from each CTA) by 256 rows of A (of which each CTA holds 128 in shared memory,
// the MMA reads both halves), so that a CTA moves two thirds of the operand bytes
// per flop of a 128 x 256 single-CTA tile, from L2 and out of shared memory.
//
// The scale factors go from shared memory to TMEM through registers (four writer
// warps, one per lane quarter, tcgen05.st), not by tcgen05.cp: the copies queue
// with the MMAs and cost about 85 cycles each, six per step of 512 MMA cycles
// (single CTAs, 16640 x 5120 x 8192: 495 us with six copies a step, 403 with two,
// 325 with none).
//
// Roles, per CTA of the cluster of two (rank 0 = leader), 16 warps:
//   warps 0, 3   TMA producers of B^T / of A, per step (512 K): this CTA's 128 rows
//                of the operand (128-byte swizzle, two 128-byte halves), completing
//                on the leader's stage barrier, and the scale tiles of its rows of
//                B^T / of all 256 rows of A, completing on its own.
//   warp 1       TMEM allocation (both CTAs); in the leader, lane 0 issues the
//                pair MMAs, eight 256x256x64 per step.
//   warps 4-11   epilogue: warp w reads lanes 32 (w % 4) .. +31 and 128 of the
//                256 columns into registers, releases the accumulator,
//                converts and stores.
//   warps 12-15  scale-factor writers.
// A stage's TMEM scale columns are written again only after the MMAs that read
// them have completed: the writers follow a refill, which follows the commit.
// TMEM: the 256-column accumulator, then kF4PairStages x 48 scale columns.
//
// 16640 x 5120 x 8192 takes 226-242 us (5.8-6.2 PFLOP/s; the tensor pipe is busy 86%
// of the time) and 270 in a long row of calls, under the power cap.  A tile's
// fixed 1.5 us (the accumulator's way out before the next tile may start: TMEM
// has no room for a second one beside the scale factors) is what short K pays.
//
// Every wait is bounded as in gemm_pair_kernel.cuh; a wait that runs out stops
// both CTAs' roles.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "ptx_fp4.cuh"
#include "mx4.cuh"
#include "gemm_kernel.cuh"
#include "gemm_pair_kernel.cuh"
#include "gemm_fp4_kernel.cuh"

namespace fp8bs {

constexpr int kF4Pair = 256;                    // rows of B^T and of A per tile
constexpr int kF4PairStepK = 512;               // K per step
constexpr int kF4PairStages = 3;
constexpr uint32_t kF4PairHalf = 128 * 128;     // one operand's 128 rows x 128 bytes (256 K)
constexpr uint32_t kF4PairTile = 2 * kF4PairHalf;
constexpr uint32_t kF4PairSf = 3 * 4 * kSfTileBytes;   // B^T's block, A's two blocks, four tiles (128 K each) each
constexpr uint32_t kF4PairSfCols = 48;
constexpr int kF4PairEpiWarps = 8;
constexpr int kF4PairThreads = 32 * (4 + kF4PairEpiWarps + 4);
constexpr int kF4LaunchRegs = 128;              // registers per thread at launch (65536 / kF4PairThreads)
constexpr int kF4CtrlRegs = 72;                 // after the hand-over: warps 0-3,
constexpr int kF4WriterRegs = 88;               // scale-factor writers,
constexpr int kF4EpiRegs = 176;                 // epilogue
static_assert(kF4Pair + kF4PairStages * kF4PairSfCols <= kTmemCols, "scale factors exceed TMEM");

struct Fp4PairSmem {
    static constexpr uint32_t w_off = 0;
    static constexpr uint32_t t_off = w_off + kF4PairStages * kF4PairTile;
    static constexpr uint32_t sf_off = t_off + kF4PairStages * kF4PairTile;
    static constexpr uint32_t bar_off = sf_off + kF4PairStages * kF4PairSf;
    // ab_full[S] (operands landed, scale columns written), ab_empty[S], sl_full[S] (scale tiles landed), tm_full, tm_empty, drain
    static constexpr uint32_t n_bars = 3 * kF4PairStages + 3;
    static constexpr uint32_t misc_off = bar_off + n_bars * 8;
    static constexpr uint32_t alloc = misc_off + 16 + 1024;
};
static_assert(Fp4PairSmem::alloc <= 232448, "shared memory per CTA");

__global__ void __launch_bounds__(kF4PairThreads, 1)
gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                     const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmST,
                     const Fp4Params p)
{
    using S = Fp4PairSmem;
    constexpr int kStages = kF4PairStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + S::bar_off;
    auto ab_full = [&](int s) { return bars + 8u * s; };
    auto ab_empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto sl_full = [&](int s) { return bars + 8u * (2 * kStages + s); };
    const uint32_t tm_full = bars + 8u * (3 * kStages);
    const uint32_t tm_empty = tm_full + 8u;
    const uint32_t drain_bar = tm_full + 16u;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + S::misc_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::misc_off + 4);
    const uint32_t abort_addr = sbase + S::misc_off + 4;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int64_t cluster_id = blockIdx.x >> 1;
    const int64_t num_clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(ab_full(s), 2 + 2 * 4);          // the leader's producers and both CTAs' writer warps
            mbar_init(ab_empty(s), 1);
            mbar_init(sl_full(s), 2);
        }
        mbar_init(tm_full, 1);
        mbar_init(tm_empty, 2 * kF4PairEpiWarps);      // both CTAs' epilogue warps
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if ((warp == 0 || warp == 3) && lane == 0) {
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmT);
        prefetch_tensormap(&tmSW);
        prefetch_tensormap(&tmST);
    }
    if (warp == 1) {
        tmem_alloc_pair(sbase + S::misc_off, kTmemCols);
        tmem_relinquish_pair();
    }
    // both CTAs' barriers initialised and TMEM allocated before anything of the
    // peer's arrives
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_begin();

    auto give_up = [&]() {
        *abort_flag = 1;
        st_shared_cluster_u32(mapa_shared(abort_addr, rank ^ 1u), 1u);
        atomicOr(p.err, 1);
    };

    // register hand-over: the launch's 128 a thread go to the epilogue's two
    // warpgroups, whose 128 accumulator columns a thread stay in registers
    static_assert(128 * (kF4CtrlRegs + kF4WriterRegs) + 256 * kF4EpiRegs <= kF4PairThreads * kF4LaunchRegs, "register hand-over");
    if (warp < 4) {
        setmaxnreg_dec<kF4CtrlRegs>();
        if (warp == 0 || warp == 3) {
            // ---------------------------------------------------------------- producers (B^T, A)
            if (lane == 0) {
                const bool wside = warp == 0;
                const CUtensorMap* map = wside ? &tmW : &tmT;
                const CUtensorMap* smap = wside ? &tmSW : &tmST;
                const uint32_t dst0 = sbase + (wside ? S::w_off : S::t_off);
                const uint32_t sf0 = sbase + S::sf_off + (wside ? 0u : 4 * kSfTileBytes);
                const uint32_t sf_bytes = (wside ? 4u : 8u) * kSfTileBytes;
                bool ok = true;
                uint32_t filled = 0, fill_par = 0;     // per stage: ever filled, parity of its latest fill
                int stage = 0;
                uint32_t phase = 0;
                for (int64_t u = cluster_id; u < p.num_units && ok; u += num_clusters) {
                    int tm, tn, split;
                    fp4_unit(p, (uint32_t)u, tm, tn, split);
                    const int tile = wside ? tn : tm;
                    const int row0 = tile * kF4Pair + (int)rank * 128;     // this CTA's rows of the operand
                    // scale tiles: of this CTA's rows of B^T, of all the tile's rows of A
                    const int block = wside ? row0 >> 7 : tile * 2;
                    for (int st = 0; st < p.steps; ++st) {
                        if (!mbar_wait_limit(ab_empty(stage), phase ^ 1u, abort_flag, kWaitLimitNs)) { ok = false; break; }
                        if (leader) mbar_arrive_expect_tx(ab_full(stage), 2 * kF4PairTile);
                        mbar_arrive_expect_tx(sl_full(stage), sf_bytes);
                        tma_load_2d(sf0 + stage * kF4PairSf, smap, sl_full(stage), st * 256, block);
                        const uint32_t full_leader = mapa_shared(ab_full(stage), 0);
                        const uint32_t dst = dst0 + stage * kF4PairTile;
                        tma_load_2d_pair(dst, map, full_leader, st * 256, row0);
                        tma_load_2d_pair(dst + kF4PairHalf, map, full_leader, st * 256 + 128, row0);
                        filled |= 1u << stage;
                        fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
                        if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    }
                }
                if (!ok) give_up();
                // the loads this thread issued land before the CTA exits; after an
                // abort a peer's load may target a phase the leader never armed, so
                // stray loads also get a fixed time
                for (int s = 0; s < kStages; ++s)
                    if (filled >> s & 1u) {
                        mbar_wait_bounded(sl_full(s), fill_par >> s & 1u, nullptr, kDrainLimitNs);
                        if (leader) mbar_wait_bounded(ab_full(s), fill_par >> s & 1u, nullptr, kDrainLimitNs);
                    }
                if (*abort_flag) {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < kPairAbortGraceNs) {
                    }
                }
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issuer (leader)
            if (leader && lane == 0) {
                int stage = 0;
                uint32_t phase = 0, tphase = 0;
                bool ok = true;
                for (int64_t u = cluster_id; u < p.num_units && ok; u += num_clusters) {
                    int tm, tn, split;
                    fp4_unit(p, (uint32_t)u, tm, tn, split);
                    if (!mbar_wait_limit(tm_empty, tphase ^ 1u, abort_flag, kWaitLimitNs)) { ok = false; break; }
                    for (int st = 0; st < p.steps; ++st) {
                        if (!mbar_wait_limit(ab_full(stage), phase, abort_flag, kWaitLimitNs)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sf = tmem_base + kF4Pair + (uint32_t)stage * kF4PairSfCols;
                        const uint64_t wd = smem_desc_k_sw128(sbase + S::w_off + stage * kF4PairTile);
                        const uint64_t td = smem_desc_k_sw128(sbase + S::t_off + stage * kF4PairTile);
                        const int left = p.K - st * kF4PairStepK;
                        // MMA k: 32 bytes further in the 128-byte rows, the second half after four; factor
                        // bytes 0, 1 or 2, 3 of the words of chunk k / 2
                        auto mma = [&](int k, uint32_t accum) {
                            const uint64_t step = (uint64_t)((k & 3) * 2 + (k >> 2) * (int)(kF4PairHalf >> 4));
                            const uint32_t id = (uint32_t)(k & 1) * 2u;
                            const uint32_t col = (sf + (uint32_t)(k >> 1) * (kF4PairSfCols / 4)) | (id << 30);
                            umma_f4_bs_pair(tmem_base, wd + step, td + step, idesc_e2m1_bs(kF4Pair, kF4Pair, id), col,
                                            col + 4, accum);
                        };
                        if (left >= kF4PairStepK) {
                            mma(0, st > 0 ? 1u : 0u);
#pragma unroll
                            for (int k = 1; k < 8; ++k) mma(k, 1u);
                        } else {
                            for (int k = 0; k * kF4MmaK < left; ++k) mma(k, (st > 0 || k > 0) ? 1u : 0u);
                        }
                        if (st + 1 == p.steps) umma_commit_pair_mc(tm_full, 0x3);
                        umma_commit_pair_mc(ab_empty(stage), 0x3);
                        if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    }
                    tphase ^= 1u;
                }
                if (!ok) give_up();
                // every MMA has completed (both CTAs' TMEM and shared memory) before the cluster tears down
                umma_commit_pair_mc(drain_bar, 0x1);
                mbar_wait_bounded(drain_bar, 0, nullptr, kDrainLimitNs);
            }
        }
    } else if (warp < 4 + kF4PairEpiWarps) {
        setmaxnreg_inc<kF4EpiRegs>();
        // ---------------------------------------------------------------- epilogue
        const int lq = warp & 3;
        const int col0 = ((warp - 4) >> 2) * 128;
        const uint32_t taddr = tmem_base + ((uint32_t)(lq * 32) << 16) + (uint32_t)col0;
        // 32 columns of D^T; whole chunks without a test per element (16640 x 5120 x
        // 256: 38 us; with the tests, when both were measured, 67 instead of 44)
        auto store = [&](auto* dst, const uint32_t (&r)[32], int cnt) {
            if (cnt <= 0) return;
            float v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
            fp4_store(dst, p.ldd, v, cnt);
        };
        uint32_t tphase = 0;
        bool ok = true;
        for (int64_t u = cluster_id; u < p.num_units; u += num_clusters) {
            int tm, tn, split;
            fp4_unit(p, (uint32_t)u, tm, tn, split);
            if (!mbar_wait_limit(tm_full, tphase, abort_flag, kWaitLimitNs)) ok = false;
            tphase ^= 1u;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const int n = tn * kF4Pair + (int)rank * 128 + lq * 32 + lane;
            const int m0 = tm * kF4Pair + col0;
            uint32_t r0[32], r1[32], r2[32], r3[32];
            tmem_ld_32x32b_x32(taddr, r0);
            tmem_ld_32x32b_x32(taddr + 32, r1);
            tmem_ld_32x32b_x32(taddr + 64, r2);
            tmem_ld_32x32b_x32(taddr + 96, r3);
            tmem_ld_wait();
            reg_after_wait32(r0);
            reg_after_wait32(r1);
            reg_after_wait32(r2);
            reg_after_wait32(r3);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(tm_empty);
                else mbar_arrive_remote(mapa_shared(tm_empty, 0));
            }
            if (n < p.N) {
                const int cols = p.M - m0;
                if (p.out_f32) {
                    float* dst = static_cast<float*>(p.D) + (int64_t)m0 * p.ldd + n;
                    store(dst, r0, cols);
                    store(dst + 32 * p.ldd, r1, cols - 32);
                    store(dst + 64 * p.ldd, r2, cols - 64);
                    store(dst + 96 * p.ldd, r3, cols - 96);
                } else {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.D) + (int64_t)m0 * p.ldd + n;
                    store(dst, r0, cols);
                    store(dst + 32 * p.ldd, r1, cols - 32);
                    store(dst + 64 * p.ldd, r2, cols - 64);
                    store(dst + 96 * p.ldd, r3, cols - 96);
                }
            }
        }
        if (!ok && lane == 0) give_up();
    } else {
        setmaxnreg_dec<kF4WriterRegs>();
        // ---------------------------------------------------------------- scale-factor writers
        const uint32_t taddr = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + kF4Pair;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = cluster_id; u < p.num_units && ok; u += num_clusters) {
            int tm, tn, split;
            fp4_unit(p, (uint32_t)u, tm, tn, split);
            for (int st = 0; st < p.steps; ++st) {
                if (!mbar_wait_limit(sl_full(stage), phase, abort_flag, kWaitLimitNs)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // lane l: row l of each tile (its four words are rows l, l + 32, ..); chunk c of the
                // step: B^T's block, A's two blocks
                const uint32_t src = sbase + S::sf_off + stage * kF4PairSf + (uint32_t)lane * 16u;
                uint32_t r[48];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 3; ++j) {
                        const uint4 v = lds_u4(src + (4 * j + c) * kSfTileBytes);
                        r[12 * c + 4 * j] = v.x;
                        r[12 * c + 4 * j + 1] = v.y;
                        r[12 * c + 4 * j + 2] = v.z;
                        r[12 * c + 4 * j + 3] = v.w;
                    }
                const uint32_t dst = taddr + (uint32_t)stage * kF4PairSfCols;
#pragma unroll
                for (int i = 0; i < 3; ++i) tmem_st_32x32b_x16(dst + 16 * i, r + 16 * i);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(ab_full(stage));
                    else mbar_arrive_remote(mapa_shared(ab_full(stage), 0));
                }
                if (++stage == kStages) { stage = 0; phase ^= 1u; }
            }
        }
        if (!ok && lane == 0) give_up();
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

}  // namespace fp8bs
