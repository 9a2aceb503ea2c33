// Which kernel and shape the 4-bit products take for a size (k_gemm4.hip).  Host code alone.
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "qamw_w8_plan.hpp"   // kCus, thin_rows

namespace qamw {

// Tiles of several sizes, and k split over workgroups where the tiles do not fill the chip; a kernel for few rows of
// activations (thin).  Larger tiles read less from L2 for each product; smaller ones fill the chip and have shorter
// starts and ends.  The choice is the least time by a model: rounds of `slots` workgroups; a full round takes
// start + more_start + steps (step + more_step) us, for steps of a group of 256 columns, one with a share f of that
// start + more_start f + steps (step + more_step f^3);  then the operands once; where k is split, its parts are written
// and read behind a launch more.  The bytes' slopes overlap with other terms: they rank kernels, and are not rates of
// memory.
struct Plan4 {
    int tile;     // index into kTiles4, or kThin4
    int splits;   // parts of k
};
struct TileCost4 {
    int bm, bn, slots;   // slots: of 64 x 64 tiles a compute unit has two at once
    double start, more_start, step, more_step;
};
// Constants fitted to measurements on MI355X of every tile and 1 to 8 parts on 609 sizes (M from 1 to 8192, N from 64 to
// 13824, K from 256 to 13824; weights in cache and not), before the tiles' output was stored streaming.  With the kernels as
// they are now, on 854 other sizes of that range, the choice takes 1.2% longer than the best one on average, over 10% longer
// for 36 sizes, and 38% at most (profiles/gemm4_choice.txt).
constexpr TileCost4 kTiles4[] = {{256, 256, 256, 7.84, 0.93, 1.062, 0.437}, {128, 256, 256, 5.67, 0.0, 0.554, 0.309},
                                 {128, 128, 256, 3.09, 0.0, 0.398, 0.124},  {64, 256, 256, 2.61, 0.79, 0.423, 0.160},
                                 {32, 256, 256, 1.88, 0.99, 0.382, 0.054},  {64, 64, 512, 0.99, 0.78, 0.249, 0.194}};
constexpr int kTileKinds4 = sizeof(kTiles4) / sizeof(kTiles4[0]), kThin4 = kTileKinds4, kThinRows4 = 32;
constexpr double kLaunch4 = 2.03, kMemory4 = 45e6, kJoin4 = 3.18, kJoinTraffic4 = 8.19e6;   // us; bytes a us
// up to 8, 16 and 32 rows: a start, a step, the weights' bytes a us, a round of workgroups
constexpr double kThin4Cost[3][4] = {{2.70, 0.040, 8.40e6, 0.0}, {3.03, 0.035, 8.29e6, 0.18}, {3.08, 0.025, 7.71e6, 0.82}};
constexpr int64_t kMaxTiles4 = 1 << 23;   // grids of 256 threads a tile stay below 2^32

inline Plan4 plan4(int M, int N, int groups) {
    Plan4 best{0, 1};
    double least = 1e300;
    const double m = M, n = N, bytes = 136.0 * groups;   // of a row
    if (M <= kThinRows4) {
        const double* c = kThin4Cost[M <= 8 ? 0 : M <= 16 ? 1 : 2];
        const int rows = thin_rows(N);
        least = c[0] + groups * c[1] + n * bytes / c[2] + c[3] * ((N + rows - 1) / rows) / kCus;
        best.tile = kThin4;
    }
    for (int i = 0; i < kTileKinds4; ++i) {
        const TileCost4& c = kTiles4[i];
        const int64_t tiles = (((int64_t)M + c.bm - 1) / c.bm) * (((int64_t)N + c.bn - 1) / c.bn);
        if (tiles > kMaxTiles4) continue;   // of 256 x 256 tiles there are never more
        for (const int s : {1, 2, 3, 4, 6, 8}) {
            if (s > 1 && (i == 0 || tiles * s > kCus || groups / s < 2)) break;   // the largest tiles gain nothing by it
            const int64_t rounds = tiles * s / c.slots, rest = tiles * s % c.slots;
            const double part = (double)((groups + s - 1) / s), f = (double)rest / c.slots;
            double t = kLaunch4 + (double)rounds * (c.start + c.more_start + part * (c.step + c.more_step));
            if (rest) t += c.start + c.more_start * f + part * (c.step + c.more_step * f * f * f);
            t += (n + m) * bytes / kMemory4;
            if (s > 1) t += kJoin4 + s * m * n * 8 / kJoinTraffic4;
            if (t < least) {
                least = t;
                best = {i, s};
            }
        }
    }
    return best;
}

// Tiles of `bm` rows that `rows` rows in `experts` groups can need: every group's last one may be a part of one.
inline int64_t group_tiles(int rows, int experts, int bm) { return rows / bm + (experts < rows ? experts : rows); }

// Rows in groups.  What the groups are is not known here, only how many rows they have on average; tiles are counted
// for groups of that many, half a tile more for each that fills one.  The same kind of model, with its own constants
// (a tile's weights come from memory, not from the tile beside it), fitted to 929 sizes (1 to 64 rows a group and
// more, in 4 to 64 groups of equal to very different sizes), before the tiles' output was stored streaming.  With the
// kernels as they are now, on 1707 other sizes, the choice takes 2.6% longer than the best one on average, over 10% longer
// for 222 of them (of those, 83 take 16 rows at a time where 8 would be better), and 57% at most (256 x 256 tiles where
// 128 x 256 would be better, as for most of the largest losses).
struct GroupCost4 {
    int tile, bm, bn;   // tile: index into kTiles4; kThin4 and kThin4 + 1: few rows of each, 8 and 16 at a time
    double start, step, more_step;
};
constexpr GroupCost4 kGroupCost4[] = {{0, 256, 256, 8.00, 1.391, 0.490}, {1, 128, 256, 4.58, 0.536, 0.778},
                                      {3, 64, 256, 2.39, 0.409, 0.641},  {4, 32, 256, 1.87, 0.355, 0.527},
                                      {kThin4, 8, 32, 1.04, 0.050, 0.054}, {kThin4 + 1, 16, 32, 1.44, 0.063, 0.058}};
constexpr double kGroupMemory4 = 33.6e6;

inline int plan4_grouped(int rows, int experts, int N, int groups) {
    const double used = experts < rows ? experts : rows, each = rows / used, g = groups;
    int best = 0;
    double least = 1e300;
    for (const GroupCost4& c : kGroupCost4) {
        const int64_t cols = ((int64_t)N + c.bn - 1) / c.bn;
        if (group_tiles(rows, experts, c.bm) * cols > kMaxTiles4) continue;   // never more of the largest
        const double tiles = used * (each <= 0.5 * c.bm ? 1.0 : each / c.bm + 0.5) * (double)cols, r = tiles / kCus;
        double t = used * N * 136.0 * g / kGroupMemory4;
        if (c.tile >= kThin4) {
            t += r * c.start + g * c.step + r * g * c.more_step;
        } else {
            const double up = (double)(int64_t)r + ((double)(int64_t)r < r), rounds = up > 1.0 ? 0.5 * (up + r) : 1.0;
            t += rounds * (c.start + g * c.step) + (r < 1.0 ? r * r * r : r) * g * c.more_step;
        }
        if (t < least) {
            least = t;
            best = c.tile;
        }
    }
    return best;
}

}  // namespace qamw
