// Product of 8-bit matrices: y[m][n] = xs_m ws_n sum_k xq[m][k] wq[n][k], exact 32-bit integer sums on
// the matrix cores (v_mfma_i32_16x16x64_i8).
//
// Both operands have their columns k contiguous.  An operand of the instruction is 16 consecutive bytes
// of one row a lane; which k a byte belongs to does not matter as long as both operands agree, so the
// rows are used as they are stored.
#include "qamw_device.hpp"
#include "qamw_w8_launch.hpp"

namespace qamw {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64, kStep = 64;

// 16 bytes of a row from column k on; zeros past the row's end or for rows that are not there.
__device__ __forceinline__ i32x4 load16(const int8_t* base, int64_t row, int rows, int64_t ld, int k, int K) {
    i32x4 v = {0, 0, 0, 0};
    if (row < rows && k < K) {
        v = *reinterpret_cast<const i32x4*>(base + row * ld + k);
#pragma unroll
        for (int d = 0; d < 4; ++d) {   // bytes past K are not part of the row
            const int left = K - k - 4 * d;
            if (left < 4) v[d] = left <= 0 ? 0 : v[d] & ((1u << (8 * left)) - 1);
        }
    }
    return v;
}

template <bool BF>
__device__ __forceinline__ void store_y(void* y, int64_t at, int c, float xs, float ws) {
    const float r = (float)c * xs * ws;
    if constexpr (BF)
        reinterpret_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)r);
    else
        reinterpret_cast<float*>(y)[at] = r;
}

// 64 x 64 tile, 4 wavefronts of 16 rows by 64 columns each.
template <bool BF>
__global__ __launch_bounds__(256) void k_gemm8(Gemm8Args a, int tiles_n) {
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kTile, n0 = (int64_t)(blockIdx.x % tiles_n) * kTile;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, r = lane % 16, g = lane / 16;
    i32x4 acc[4] = {};
    for (int k = 0; k < a.K; k += kStep) {
        const i32x4 x = load16(a.xq, m0 + wave * 16 + r, a.M, a.ld_x, k + g * 16, a.K);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const i32x4 w = load16(a.wq, n0 + c * 16 + r, a.N, a.ld_w, k + g * 16, a.K);
            acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, w, acc[c], 0, 0, 0);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + wave * 16 + 4 * g + i, n = n0 + c * 16 + r;
            if (m < a.M && n < a.N) store_y<BF>(a.y, m * a.ld_y + n, acc[c][i], a.xs[m], a.ws[n]);
        }
}

}  // namespace

size_t gemm8_workspace(int, int, int) { return 0; }

hipError_t launch_gemm8(const Gemm8Args& a, hipStream_t st) {
    const int64_t tiles_m = ((int64_t)a.M + kTile - 1) / kTile, tiles_n = ((int64_t)a.N + kTile - 1) / kTile;
    const int64_t slab = (1 << 22) / tiles_n;   // row tiles a launch: the grid stays below 2^32 work items
    for (int64_t m = 0; m < tiles_m; m += slab) {
        Gemm8Args s = a;
        const int64_t tiles = tiles_m - m < slab ? tiles_m - m : slab, rows = (int64_t)a.M - m * kTile;
        s.xq += m * kTile * a.ld_x;
        s.xs += m * kTile;
        s.M = (int)(rows < tiles * kTile ? rows : tiles * kTile);
        s.y = reinterpret_cast<char*>(a.y) + m * kTile * a.ld_y * (a.y_bf16 ? 2 : 4);
        const dim3 grid((unsigned)(tiles * tiles_n));
        if (a.y_bf16)
            hipLaunchKernelGGL((k_gemm8<true>), grid, dim3(256), 0, st, s, (int)tiles_n);
        else
            hipLaunchKernelGGL((k_gemm8<false>), grid, dim3(256), 0, st, s, (int)tiles_n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qamw
