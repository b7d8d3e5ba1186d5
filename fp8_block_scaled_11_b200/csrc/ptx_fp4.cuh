// ptx_fp4.cuh -- inline-PTX wrappers of the 4-bit block-scaled MMA (sm_100a) and
// of the untiled bulk copy that brings its scale tiles.  Single instructions, as
// in ptx.cuh.
#pragma once

#include <cstdint>
#include "ptx.cuh"
#include "ptx_bs.cuh"

namespace fp8bs {

// kind::mxf4.block_scale, scale_vec::2X: E2M1 x E2M1 -> F32, K = 64 per
// instruction, one UE8M0 factor per 32 K.  Instruction descriptor: bits [4,6)
// the B scale-factor id, [7,10) the A format (E2M1 = 1), [10,12) the B format,
// 15 / 16 A / B major (K = 0), [17,23) N >> 3, bit 23 the scale type (1 =
// UE8M0), [27,29) M >> 7, [29,31) the A scale-factor id, bit 31 the K size (0 =
// 64).  The id (0 or 2) names the first of the two bytes of each 32-bit TMEM
// scale-factor word that this MMA uses.
__host__ __device__ constexpr uint32_t idesc_e2m1_bs(uint32_t M, uint32_t N, uint32_t sf_id)
{
    return (sf_id << 4)
         | (1u << 7) | (1u << 10)
         | (0u << 15) | (0u << 16)
         | ((N >> 3) << 17)
         | (1u << 23)
         | ((M >> 7) << 27)
         | (sf_id << 29);
}

// D[tmem] (+)= (A[smem] . B[smem]^T), each product of 32 K scaled by its rows'
// factors at sfa / sfb in TMEM (the byte id also in bits [30,32) of these
// addresses).
__device__ __forceinline__ void umma_f4_bs(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
        : "memory");
}

// The pair form (issued by the leader): M = 256, 128 rows of A from each CTA's
// shared memory, half of B's rows from each; every CTA's TMEM holds its own rows
// of the accumulator, its own rows' factors at sfa and all of B's at sfb.
__device__ __forceinline__ void umma_f4_bs_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t sfa, uint32_t sfb, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
        : "memory");
}

// Programmatic launches: waits until the kernels before this one have completed
// and their results are visible, then lets the next one be set up on SMs with
// room; before it no kernel touches memory that another may write.
__device__ __forceinline__ void grid_begin()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The 128-byte line at p into L2 only, which stays coherent: allowed before
// grid_begin whoever writes the data.
__device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Thread i of the warp writes 16 consecutive columns of TMEM lane
// lane_base + i; complete after tmem_st_wait.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_nctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// The two halves of a cluster barrier: work between them runs while the peers
// arrive.  Every thread of the CTA executes both.  The arrival orders no memory
// (a releasing one cost 800 cycles here): what the peers may use are mbarriers,
// published by fence_barrier_init.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A float of a cluster CTA's shared memory.
__device__ __forceinline__ float lds_cluster(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// 16 bytes into a cluster CTA's shared memory, counted on an mbarrier of the
// same CTA (both shared::cluster addresses).
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, const uint32_t* r, uint32_t cluster_bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(cluster_addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(cluster_bar)
                 : "memory");
}

// mbar_wait_bounded that looks at the clock only every 64 tries (each try waits
// inside the instruction for a while): the tries that find the phase complete,
// nearly all of them, read no timer.
__device__ __forceinline__ bool mbar_wait_limit(uint32_t bar, uint32_t parity, const volatile int* abort,
                                                uint64_t limit_ns)
{
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0u) {
            if (abort != nullptr && *abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > limit_ns) return false;
        }
    }
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned,
// counted on mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

}  // namespace fp8bs
