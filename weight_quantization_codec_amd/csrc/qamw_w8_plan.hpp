// Which kernel and shape the 8-bit product takes for a size (k_gemm8.hip).  Host code alone.
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace qamw {

constexpr int kCus = 256;

// Weight rows of a workgroup: at most 32, and the same for all workgroups of all rounds over the compute
// units (20 of 5120 rows: 256 workgroups).
inline int thin_rows(int n) {
    const int64_t wgs = (((int64_t)n + kCus * 32 - 1) / (kCus * 32)) * kCus;
    const int rows = (int)((n + wgs - 1) / wgs);
    return rows < 8 ? 8 : rows;
}

// Tiles of several sizes, and k split over workgroups where the tiles do not fill the chip.  Larger tiles
// read less from L2 for each product; smaller ones fill the chip and have shorter starts and ends.  The
// choice is the least time by a model: rounds of up to 256 workgroups, one a compute unit; a round with
// a share f of that takes  start + more_start f + steps (step + more_step f^3)  us, for steps of 128 bytes of
// k; then the operands once; the sums of k's parts are written and read, behind a launch.
// The thin kernel (at most 64 activation rows) has the weights once, and the activations once a workgroup.
// The bytes' slopes are fitted like the other constants, over operands in the 256 MB cache and out of it, and next to
// terms that overlap with them: they rank kernels, and are not rates of memory (a large copy reaches 5.1 TB/s).
struct Plan {
    int tile;     // index into kTiles, or kThin
    int splits;   // parts of k
};
struct TileCost {
    int bm, bn;
    double start, more_start, step, more_step;
};
// Constants fitted to measurements on MI355X of every tile and 1 to 16 parts on 200 sizes (M from 1 to 8192, N and
// K from 64 to 13824; weights in cache and not).  There the choice takes 1% longer than the best one on average and
// 19% at most (profiles/gemm8_choice_200_sizes.txt); the largest losses are near the border of the thin kernel, whose
// time the model takes too high for one token (1 x 5120 x 5120: 8.6 us; measured 5.7 in cache, 7.9 from memory).
constexpr TileCost kTiles[] = {{256, 256, 8.9, 0.9, 0.89, 0.44}, {256, 128, 5.2, 1.1, 0.54, 0.27},
                               {128, 128, 3.6, 0.8, 0.37, 0.10}, {128, 64, 2.9, 0.9, 0.27, 0.025},
                               {64, 128, 2.5, 1.3, 0.35, 0.03},  {64, 64, 2.4, 0.4, 0.21, 0.03}};
constexpr double kLaunch = 1.3, kMemory = 28e6, kJoin = 2.9, kJoinTraffic = 8.9e6;   // us; bytes a us
constexpr double kThinStart = 3.9, kThinStep = 0.046, kThinWeights = 10.6e6, kThinActivations = 25.7e6;
constexpr int64_t kMaxTiles = 1 << 23;   // grids of 256 threads a tile stay below 2^32
constexpr int kTileKinds = sizeof(kTiles) / sizeof(kTiles[0]), kThin = kTileKinds, kThinRows = 64;

inline Plan plan(int M, int N, int K) {
    Plan best{0, 1};
    double least = 1e300;
    const double m = M, n = N, k = K;
    const int64_t steps = (K + 127) / 128;
    if (M <= kThinRows) {
        const int rows = thin_rows(N);
        const double wgs = (double)((N + rows - 1) / rows), x_rows = M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
        least = kThinStart + (double)steps * kThinStep + n * k / kThinWeights + wgs * x_rows * k / kThinActivations;
        best.tile = kThin;
    }
    for (int i = 0; i < kTileKinds; ++i) {
        const TileCost& c = kTiles[i];
        const int64_t tiles = (((int64_t)M + c.bm - 1) / c.bm) * (((int64_t)N + c.bn - 1) / c.bn);
        if (tiles > kMaxTiles) continue;   // of 256 x 256 tiles there are never more
        for (const int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (s > 1 && (i == 0 || tiles * s > kCus || steps / s < 3)) break;   // the largest tiles gain nothing by it
            const int64_t rounds = tiles * s / kCus, rest = tiles * s % kCus;
            const double part = (double)((steps + s - 1) / s), f = (double)rest / kCus;
            double t = kLaunch + (double)rounds * (c.start + c.more_start + part * (c.step + c.more_step));
            if (rest) t += c.start + c.more_start * f + part * (c.step + c.more_step * f * f * f);
            t += (n * k + m * k) / kMemory;
            if (s > 1) t += kJoin + s * m * n * 8 / kJoinTraffic;
            if (t < least) {
                least = t;
                best = {i, s};
            }
        }
    }
    return best;
}

}  // namespace qamw
