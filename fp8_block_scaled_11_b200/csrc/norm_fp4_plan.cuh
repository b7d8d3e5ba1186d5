// norm_fp4_plan.cuh -- which kernel, tile and split a 4-bit product takes, and its
// workspace.  Host code.
#pragma once

#include <algorithm>
#include <cstdint>
#include "gemm_fp4_kernel.cuh"
#include "gemm_fp4_pair_kernel.cuh"

namespace fp8bs {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
