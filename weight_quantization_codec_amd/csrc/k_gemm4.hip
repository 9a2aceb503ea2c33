// Products of matrices of 4-bit codes with a power of two for every 32 columns: y[m][n] = sum_k x[m][k] w[n][k], on
// the matrix cores (v_mfma_scale_f32_32x32x64_f8f6f4), and the same for rows in groups with weights of their own.
//
// An operand of the instruction is one block of 32 columns a lane, with the block's scale byte: lane l has row l % 32,
// and lanes 0-31 and 32-63 have two different blocks.  Which blocks does not matter as long as both operands agree:
// of a group of 8 blocks the lower lanes have 0-3 and the upper ones 4-7, so that a lane's four scale bytes are
// the four bytes of a register, from which the instruction takes the one that it is told.
#include "qamw_device.hpp"
#include "qamw_mx4_launch.hpp"
#include "qamw_rows.hpp"
#include "qamw_tile.hpp"

namespace qamw {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// acc += the products of two blocks a row, scale byte B of sw and sx.
template <int B>
__device__ __forceinline__ f32x16 mfma4(i32x4 w, i32x4 x, f32x16 acc, int sw, int sx) {
    constexpr int kFp4 = 4;
    const i32x8 w8 = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 x8 = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x8, acc, kFp4, kFp4, B, sw, B, sx);
}

// Rows in groups: the expert and the rows of the tile `tile` of `bm` rows, counted over all groups; false past the
// last tile.  Every lane of the wavefront calls this.
__device__ __forceinline__ int clamped(const int32_t* offsets, int e, int rows) {
    const int o = offsets[e];
    return o < 0 ? 0 : o > rows ? rows : o;
}
__device__ __forceinline__ bool group_tile(const Gemm4Args& a, int bm, int tile, int& expert, int& first, int& end) {
    const int lane = threadIdx.x % kWave;
    for (int e0 = 0; e0 < a.experts; e0 += kWave) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.experts) {
            lo = clamped(a.offsets, e, a.M);
            hi = clamped(a.offsets, e + 1, a.M);
        }
        const int tiles = hi > lo ? (hi - lo + bm - 1) / bm : 0;
        int sum = tiles;   // of this lane's groups and all before it
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const int below = __shfl_up(sum, off);
            sum += lane >= off ? below : 0;
        }
        const uint64_t reached = __ballot(sum > tile);
        if (reached) {
            const int at = __builtin_ctzll(reached);
            expert = e0 + at;
            first = __shfl(lo, at) + (tile - __shfl(sum - tiles, at)) * bm;
            end = __shfl(hi, at);
            return true;
        }
        tile -= __shfl(sum, kWave - 1);
    }
    return false;
}

// The simplest form: a wavefront has 32 rows of y and 32 columns, and loads its operands as they stand in memory.
template <bool GROUPED>
__device__ __forceinline__ void tile_simple(const Gemm4Args& a, int tile_m, int n0) {
    const int lane = threadIdx.x % kWave, r = lane % 32, h = lane / 32;
    int expert = 0, m0 = tile_m * 32, m_end = a.M;
    if (GROUPED && !group_tile(a, 32, tile_m, expert, m0, m_end)) return;
    const int n = n0 + r < a.N ? n0 + r : a.N - 1, m = m0 + r < m_end ? m0 + r : m_end - 1;
    int row = m;
    if (GROUPED && a.index) row = a.index[m];
    const bool none = GROUPED && (row < 0 || row >= a.x_rows);
    const uint8_t* x = a.xq + row * a.ld_x + h * 64;
    const uint8_t* xe = a.xe + row * 8ll + h * 4;
    const uint8_t* w = a.wq + (GROUPED ? expert * a.ld_wexpert : 0) + n * a.ld_w + h * 64;
    const uint8_t* we = a.we + (GROUPED ? expert * a.ld_weexpert : 0) + n * 8ll + h * 4;
    f32x16 acc = (f32x16)(0.0f);
    for (int g = 0; g < a.groups; ++g) {
        const int sx = none ? 0 : *reinterpret_cast<const int*>(xe + g * a.ld_xe);
        const int sw = *reinterpret_cast<const int*>(we + g * a.ld_we);
        static_for<4>([&](auto b) {
            i32x4 fx = (i32x4)(0);
            if (!none) fx = *reinterpret_cast<const i32x4*>(x + g * kGroupBytes + b * 16);
            const i32x4 fw = *reinterpret_cast<const i32x4*>(w + g * kGroupBytes + b * 16);
            acc = mfma4<b>(fw, fx, acc, sw, sx);
        });
    }
    if (m0 + r >= m_end) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int col = n0 + i / 4 * 8 + h * 4 + i % 4;
        if (col >= a.N) continue;
        const int64_t at = (int64_t)m * a.ld_y + col;
        if (a.y_bf16)
            reinterpret_cast<uint16_t*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)acc[i]);
        else
            reinterpret_cast<float*>(a.y)[at] = acc[i];
    }
}

template <bool GROUPED>
__global__ __launch_bounds__(256) void k_gemm4_simple(Gemm4Args a, int tiles_m) {
    const int tiles_n = (a.N + 31) / 32;
    const int64_t all = (int64_t)tiles_m * tiles_n;
    for (int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; t < all; t += (int64_t)gridDim.x * 4)
        tile_simple<GROUPED>(a, (int)(t / tiles_n), (int)(t % tiles_n) * 32);
}

template <bool GROUPED>
hipError_t launch_simple(const Gemm4Args& a, int tiles_m, hipStream_t st) {
    const int64_t wgs = ((int64_t)tiles_m * ((a.N + 31) / 32) + 3) / 4, most = 1 << 20;
    return launch_kernel(k_gemm4_simple<GROUPED>, dim3((unsigned)(wgs < most ? wgs : most)), 256, 0, st, a, tiles_m);
}

}  // namespace

size_t gemm4_workspace(int, int, int) { return 0; }

hipError_t launch_gemm4(const Gemm4Args& a, hipStream_t st) { return launch_simple<false>(a, (a.M + 31) / 32, st); }

hipError_t launch_gemm4_grouped(const Gemm4Args& a, hipStream_t st) {
    // every group's last tile may be a part of one
    return launch_simple<true>(a, a.M / 32 + (a.experts < a.M ? a.experts : a.M), st);
}

}  // namespace qamw
