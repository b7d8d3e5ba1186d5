// norm_fp4_plan.cuh -- which kernel, threads, tile and split the RMS norm, its
// backward pass and the 4-bit product take, and their workspaces.  Host code.
#pragma once

#include <algorithm>
#include <cstdint>
#include "norm_kernels.cuh"
#include "gemm_fp4_kernel.cuh"
#include "gemm_fp4_pair_kernel.cuh"

namespace fp8bs {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int64_t round32(int64_t v) { return (v + 31) / 32 * 32; }

// ---------------------------------------------------------------- RMS norm
// Threads per row (16, or a multiple of 32) and eights per thread for a row of
// `eights` eights: the pair that leaves the fewest threads idle, at most max_tx
// threads; among equals the first of `order`.
struct RowShape {
    int tx, vpt;                // vpt == 0: the row is too wide
};

inline int64_t round_row(int64_t tx) { return tx <= 16 ? 16 : round32(tx); }

inline RowShape row_shape(int64_t eights, int64_t max_tx, const int (&order)[3])
{
    RowShape best = {0, 0};
    int64_t best_idle = INT64_MAX;
    for (int vpt : order) {
        const int64_t tx = round_row(cdiv(eights, vpt));
        if (tx <= max_tx && tx * vpt - eights < best_idle) {
            best_idle = tx * vpt - eights;
            best = {(int)tx, vpt};
        }
    }
    return best;
}

// The backward's launches and the bytes of its workspace.  Rows are read once, over
// a ring, where two slots of one row fit and 512 threads hold it: up to 16384
// columns of bf16; of fp32 up to 14128, with dh 9424.  That is two launches (the
// second adds up dweight), or one where a cluster takes all rows.  Wider rows take
// three: their dot products, dx, dweight.
struct BackPlan {
    RowShape shape;             // vpt == 0: wide rows
    int ty, slots, per_sm;      // rows per block of the ring, its depth, CTAs per SM
    int cluster;                // CTAs of the one cluster that takes all rows (0: many CTAs, and a second launch)
    uint32_t smem;
    int64_t grid, parts;
    size_t dot_off, bytes;
};

constexpr uint32_t kRingSmem = 222 * 1024;      // of an SM's shared memory
constexpr int kBackCluster = 8;                 // CTAs of a cluster, at most

inline BackPlan plan_back(int64_t rows, int64_t cols, int64_t elem, int mats, int num_sms)
{
    BackPlan b = {};
    const int64_t eights = cdiv(cols, 8);
    const uint32_t row_bytes = (uint32_t)std::min<int64_t>(cols * elem, kRingSmem);
    // eights per thread: one where 16 threads hold a row (100000 x 128 bf16 21 us, with
    // two 26), over 1024 threads of an SM; else four or two over 512, whichever keeps
    // more of them at work.  Among equals four (16640 x 1616 bf16 39 us, with two 47),
    // but two where the SMs have under three rows each, whose latency counts (161 x
    // 3776 bf16 6.0 us, with four 6.2; 333 x 1040 fp32 5.8 and 6.4).  A CTA has 256
    // threads (or one row's) and room for two slots.
    double best = 0.;
    for (int i = 0; i < 2; ++i) {
        const bool narrow = eights <= 16;
        const bool two_first = rows < 3 * num_sms && eights <= 512;     // (at most 256 threads a row)
        const int vpt = narrow ? 1 : two_first == (i == 0) ? 2 : 4;
        const int64_t tx = narrow ? 16 : round_row(cdiv(eights, vpt));
        if (tx > 512) continue;
        int ty = std::max(1, (int)(256 / tx));
        while (ty > 1 && cdiv(rows, ty) < num_sms) ty /= 2;             // few rows: over more SMs
        if (tx == 16) ty = (ty + 1) / 2 * 2;                            // whole warps
        const uint32_t slot = ring_smem(row_bytes, ty, mats, 1);
        const int per_sm = (int)std::min<int64_t>((narrow ? 1024 : 512) / (tx * ty), kRingSmem / (2 * slot + 1024));
        const double busy = (double)per_sm * (double)ty * (double)eights / vpt;
        if (per_sm < 1 || busy <= best) continue;
        best = busy;
        b.shape = {(int)tx, vpt};
        b.ty = ty;
        b.per_sm = per_sm;
        b.slots = (int)std::min<uint32_t>(4, (kRingSmem / (uint32_t)per_sm - 1024) / slot);
        b.smem = ring_smem(row_bytes, ty, mats, b.slots);
    }
    if (b.shape.vpt > 0) b.grid = std::min<int64_t>(cdiv(rows, b.ty), (int64_t)b.per_sm * num_sms);
    else b.grid = std::max<int64_t>(1, std::min<int64_t>(rows, 8 * num_sms / cdiv(cols, 2048)));
    b.parts = b.grid;
    b.dot_off = (size_t)(b.parts * cols) * sizeof(float);
    b.bytes = b.dot_off + (b.shape.vpt == 0 ? (size_t)((rows + 3) / 4 * 4) * sizeof(float) : 0);
    // few narrow rows: one cluster takes them all and adds up dw itself, without the
    // second launch (64 x 512 bf16 4.0 us instead of 4.3, called from Python 4.6
    // instead of 6.2; 16 x 1024 4.5 and 4.1, 5.0 and 6.1; at 4096 columns slower)
    const int ty = b.shape.vpt > 0 ? 256 / std::min(b.shape.tx, 256) : 1;
    const int64_t blocks = cdiv(rows, ty);
    if ((b.shape.vpt == 1 || b.shape.vpt == 2) && blocks <= (b.shape.tx == 16 ? 2 : b.shape.tx <= 64 ? 1 : 0) * kBackCluster) {
        b.cluster = blocks > 4 ? kBackCluster : blocks > 2 ? 4 : (int)blocks;
        b.ty = ty;
        b.slots = 2;
        b.smem = ring_smem(row_bytes, ty, mats, 2);
        b.grid = b.cluster;
    }
    return b;
}

// ---------------------------------------------------------------- 4-bit product
struct Fp4Plan {
    bool pair;                  // 256 x 256 tiles on CTA pairs; else 128 x bn tiles on single CTAs
    int bn;
    int tiles_m, tiles_n;
    int parts;                  // CTAs of a cluster that share a tile's K
    int splits;                 // parts of K that go through the workspace
    int64_t ldw;
    size_t ws_bytes;
};

// What a product takes on single CTAs, in us: units (a tile's part of K) over SMs
// that hold two, each round of them the tile's fixed part and its steps of 256 K,
// where a round leaves an SM to each unit (`fixed`, `step`) or puts two on it
// (`fixed2`, `step2`), and what sending and adding a cluster's sums adds.
struct Fp4Cost {
    double fixed, step, fixed2, step2, send, send2;
};

inline double fp4_single_us(const Fp4Cost& c, int64_t units, int64_t steps, bool send, int num_sms)
{
    const int64_t room = 2 * num_sms, rounds = units / room, rest = units % room;
    double us = (double)rounds * (c.fixed2 + c.step2 * (double)steps);
    if (rest > num_sms) us += c.fixed2 + c.step2 * (double)steps;
    else if (rest > 0) us += c.fixed + c.step * (double)steps;
    return us + (!send ? 0. : units > num_sms ? c.send2 : c.send);
}

// Tiles and the split of K: the fastest of CTA pairs and of single CTAs with each
// tile width and cluster size, by models of their times fitted to 600 measured
// ones (M 130 .. 4096, N 1000 .. 32000, K 256 .. 8192), where the choice costs
// 0.6% over the fastest in the mean and 14% at most.  Measured: 1024 x 5120 x 8192
// 24.7 us on pairs, 31.5 on single CTAs of 128 columns; 512 x 8192 x 256 4.6 with
// 128 columns, 7.4 with 64; 256 x 2080 x 8192 10.3 with 64 columns over clusters of
// four, 13.6 on pairs; 72 x 5120 x 8192 9.0 over clusters of four, 14.2 without.
// pairs: whether CTA pairs are to be had at all.
inline Fp4Plan plan_fp4(int64_t M, int64_t N, int64_t K, int num_sms, bool pairs = true)
{
    static constexpr Fp4Cost kCost[4] = {{0.2, 0.30, 0.2, 0.30, 0.35, 0.5},       // 16 columns
                                         {0.4, 0.30, 0.4, 0.30, 0.7, 1.0},        // 32
                                         {2.1, 0.38, 2.8, 0.41, 1.3, 1.8},        // 64
                                         {2.5, 0.39, 3.3, 0.45, 2.6, 3.2}};       // 128
    Fp4Plan s = {};
    const int64_t steps = cdiv(K, kF4StepK);
    s.tiles_n = (int)cdiv(N, kF4Rows);
    s.parts = 1;
    s.splits = 1;
    double best = 1e30;
    // the narrowest tile that holds every token, or either of the two widest ones
    for (int i = M <= 16 ? 0 : M <= 32 ? 1 : 2, bn = 16 << i; i < 4; ++i, bn *= 2) {
        const int64_t units = cdiv(M, bn) * s.tiles_n;
        for (int parts = 1; parts <= kF4MaxCluster; parts *= 2) {
            if (parts > 1 && (units * parts > 2 * num_sms || steps < 2 * parts)) break;
            const double us = fp4_single_us(kCost[i], units * parts, cdiv(steps, parts), parts > 1, num_sms);
            if (us < best) {
                best = us;
                s.bn = bn;
                s.parts = parts;
            }
        }
        if (M <= bn) break;
    }
    const int64_t waves = cdiv(cdiv(M, kF4Pair) * cdiv(N, kF4Pair), std::max(1, num_sms / 2));
    s.pair = pairs && M > 128 && 2.85 + (double)waves * (1.48 + 0.308 * (double)steps) < best;
    if (s.pair) {
        s.bn = kF4Pair;
        s.tiles_n = (int)cdiv(N, kF4Pair);
        s.parts = 1;
    } else {
        // very long K over clusters too, where they leave half of the room and 8 steps a CTA
        const int64_t ctas = cdiv(M, s.bn) * s.tiles_n * s.parts;
        if (s.parts == kF4MaxCluster)
            s.splits = (int)std::max<int64_t>(1, std::min<int64_t>({2 * num_sms / ctas, steps / (8 * s.parts), 32}));
    }
    s.tiles_m = (int)cdiv(M, s.bn);
    s.ldw = (N + 3) & ~int64_t(3);
    s.ws_bytes = s.splits > 1 ? (size_t)s.splits * (size_t)M * (size_t)s.ldw * sizeof(float) : 0;
    return s;
}

}  // namespace fp8bs
