// Which kernel and shape the 4-bit products take for a size (k_gemm4.hip).  Host code alone.
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "qamw_w8_plan.hpp"   // kCus, thin_rows

namespace qamw {

// Tiles of several sizes, and k split over workgroups where the tiles do not fill the chip; a kernel for few rows of
// activations (thin).  The choice is the least time by a model: rounds of up to 256 workgroups, one a compute unit,
// each  start + steps step  us for steps of a group of 256 columns; where k is split, its parts are written, read and
// added behind one launch more.
struct Plan4 {
    int tile;     // index into kTiles4, or kThin4
    int splits;   // parts of k
};
struct TileCost4 {
    int bm, bn;
    double start, step;
};
constexpr TileCost4 kTiles4[] = {{256, 256, 7.5, 1.5}, {128, 256, 5.0, 0.80}, {128, 128, 3.5, 0.50},
                                 {64, 256, 4.0, 0.55}, {32, 256, 3.5, 0.45},  {64, 64, 3.0, 0.31}};
constexpr int kTileKinds4 = sizeof(kTiles4) / sizeof(kTiles4[0]), kThin4 = kTileKinds4, kThinRows4 = 32;
constexpr double kLaunch4 = 1.3, kJoin4 = 2.9, kJoinTraffic4 = 8.9e6;   // us; bytes a us
constexpr double kThinStart4 = 2.5, kThinWeights4 = 5.0e6, kThinActivations4 = 12e6;
constexpr int64_t kMaxTiles4 = 1 << 23;   // grids of 256 threads a tile stay below 2^32

inline Plan4 plan4(int M, int N, int groups) {
    Plan4 best{0, 1};
    double least = 1e300;
    const double m = M, n = N, bytes = 136.0 * groups;   // of a row
    if (M <= kThinRows4) {
        const int rows = thin_rows(N);
        const double wgs = (double)((N + rows - 1) / rows), x_rows = M <= 8 ? 8 : M <= 16 ? 16 : 32;
        least = kLaunch4 + kThinStart4 + n * bytes / kThinWeights4 + wgs * x_rows * bytes / kThinActivations4;
        best.tile = kThin4;
    }
    for (int i = 0; i < kTileKinds4; ++i) {
        const TileCost4& c = kTiles4[i];
        const int64_t tiles = (((int64_t)M + c.bm - 1) / c.bm) * (((int64_t)N + c.bn - 1) / c.bn);
        if (tiles > kMaxTiles4) continue;   // of 256 x 256 tiles there are never more
        for (const int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (s > 1 && (i == 0 || tiles * s > kCus || groups / s < 3)) break;   // the largest tiles gain nothing by it
            const double rounds = (double)((tiles * s + kCus - 1) / kCus), part = (double)((groups + s - 1) / s);
            double t = kLaunch4 + rounds * (c.start + part * c.step);
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

// Rows in groups: what the groups are is not known here, only how many rows they have on average.  A tile of 256
// columns keeps enough of the weights on their way, whatever its rows, and takes its rows from one group.
inline int plan4_grouped(int rows, int experts, int N) {
    const double each = (double)rows / experts;
    if (rows <= 16 && (int64_t)rows * N < 256 * 256) return kThin4;
    for (const int kind : {4, 3, 1}) {
        const TileCost4& c = kTiles4[kind];
        const int64_t tiles = group_tiles(rows, experts, c.bm) * (((int64_t)N + c.bn - 1) / c.bn);
        if (each <= (kind == 4 ? 6 : kind == 3 ? 100 : 200) && tiles <= kMaxTiles4) return kind;
    }
    return 0;   // never more than kMaxTiles4, by the limits of the sizes
}

}  // namespace qamw
