// i8_plan.h -- which tile, and how many runs of the sum, the int8 products and gradients take.
// Host only.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "tile_rounds.h"

namespace gq {

// The tile for a shape, from an estimate of its time: stages (128 columns) in full rounds of
// tiles on the device and a last one by how many CUs it has, and what a round takes besides.
// Measured, us for K 14336 (112 stages): 64 x 64 tiles 26 up to one per CU, 46 at two, 92 at
// four; 128 x 128 47 alone, 66 at one per CU; 256 x 256 67 for a lone round in halves, 194 a full
// round.  So 4096 x 14336 takes by 130 rows 26 us on the first (47, 67 on the others), by 1024
// rows 66 on the second (93, 81), by 4096 rows 194 on the third (356, 252); 1003 x 2048 by 77
// rows 6.2, 11.3 and 14.5, 4096 x 512 by 1024 rows 9.9, 8.1 and 8.8.  Gate/up, whose smallest
// tiles are 128 x 64: 14336 x 4096 by 64 rows 21, 28 and 29, by 130 rows 44, 47 and 37.
inline int i8_tile_choice(int64_t M, int64_t K, int64_t N, bool pair, int64_t cus)
{
    const double st = (double)((K + 127) / 128);
    auto tiles = [&](int64_t m, int64_t n) { return (M + m - 1) / m * ((N + n - 1) / n); };
    auto last = [&](int64_t rest, double lone, double full) {
        return rest ? lone + (full - lone) * (double)rest / (double)cus : 0;
    };
    auto rounds = [&](int64_t t) { return 2.5 * (double)((t + cus - 1) / cus); };
    const int64_t t2 = tiles(128, 128), t3 = tiles(256, 256), whole = tiles_whole(t3, cus);
    const double per_cu = (double)(pair ? tiles(128, 64) : tiles(64, 64)) / (double)cus;
    const double more = std::max(0.0, per_cu - 1.0);
    const double t64 = st * (pair ? 0.25 + 0.3 * std::min(per_cu, 1.0) + 0.4 * more : 0.2 + 0.195 * more) + 1.1 * more;
    const double t128 = st * (0.58 * (double)(t2 / cus) + last(t2 % cus, 0.42, 0.58)) + rounds(t2);
    const double t256 = st * (1.72 * (double)(t3 / cus) +
                              (whole < t3 ? last(2 * (t3 - whole), 0.6, 1.15) : last(t3 % cus, 1.2, 1.72))) +
                        rounds(t3);
    return t64 <= t128 && t64 <= t256 ? 64 : t128 <= t256 ? 128 : 256;
}

struct GradTile {
    int columns, rows, per_cu; // of a tile, and tiles a CU holds
    double stage[3];           // us a stage takes with one, two, three of them on every CU
};
constexpr GradTile kGradTiles[] = {{256, 256, 1, {1.8}}, {256, 128, 1, {1.25}}, {128, 64, 3, {0.8, 1.2, 1.23}}};

struct GradPlan {
    int tile, splits;
};
// The tile and the number of runs with the least estimated time: rounds of workgroups on the
// device, 1.8 us for a workgroup's start and end, stages of a round that leaves CUs idle down to
// two thirds of a full one's; runs add a launch, something each, and the traffic of their sums.
// Fitted to measurements with weights from HBM, each tile with 1 to 16 runs: over 37 sizes, eleven
// of them not fitted to, the choice is within 7% of the best measured, in 30 within 2%.  4096 x
// 4096, us, the best number of runs of each tile: by 16 rows 18.8 (12 runs), 16.4 (12), 16.1 (8); by
// 130 rows 29.2 (10), 26.2 (7), 26.2 (7), in one run 90, 69, 56; by 512 rows 45.9 (5), 39.7 (4), 43.3
// (3); by 4096 rows 122, 151, 230 (1).  14336 x 4096 by 2048 rows 232 (2), 255 (1), 397 (3).  More
// than 16 runs gain 5% at most (a gated half 14336 x 4096 by one row, 24 runs), for sums half again
// as large.  256 CUs are the whole device's: the workspace, whose size this decides, is a matter of
// the sizes alone, whatever part of a device the caller sees.
inline GradPlan grad_plan(int nparts, int64_t M, int64_t K, int64_t N)
{
    constexpr int64_t kCus = 256;
    const int64_t stages = nparts * ((M + 63) / 64);
    GradPlan best{};
    double least = 1e30;
    for (int i = 0; i < 3; ++i) {
        const GradTile &t = kGradTiles[i];
        const int64_t tiles = (K + t.columns - 1) / t.columns * ((N + t.rows - 1) / t.rows);
        for (int s = 1; s <= 16 && s <= stages; ++s) {
            const int64_t full = tiles * s / (kCus * t.per_cu), rest = tiles * s % (kCus * t.per_cu);
            const double each = (double)((stages + s - 1) / s);
            double us = (double)full * (each * t.stage[t.per_cu - 1] + 1.8);
            if (rest) {
                const double part = t.per_cu > 1 ? 1.0 : 0.67 + 0.33 * (double)rest / (double)kCus;
                us += each * part * t.stage[(rest - 1) / kCus] + 1.8;
            }
            if (s > 1)
                us += 2.8 + 0.28 * s + (double)(s * N * K) * 8.0 / 5.8e6;
            if (us < least)
                least = us, best = {i, s};
        }
    }
    return best;
}

} // namespace gq
