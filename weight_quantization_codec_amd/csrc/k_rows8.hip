// Rows of a matrix as 8-bit codes with a scale each (quant8, rmsnorm8), and back (dequant8).
//
// k_rows8: one workgroup per row at a time, the row in registers: every thread holds V chunks of 8
// consecutive columns, chunk t + v * threads, so a wavefront's loads are contiguous.  One pass over
// HBM: the row's largest magnitude (and for the norm its sum of squares) is reduced over the
// workgroup, then the codes are formed from the registers.  The norm's factor 1 / rms is the same for
// the whole row, so it changes the row scale and no code: codes need the largest magnitude only, and
// both reductions share one barrier.
//
// Rounding.  Values are fp32 from the load on; the sum of squares is fp64, which holds the square of
// every fp32 value and adds 32768 of them without overflow or loss that matters.  Magnitudes are
// compared as bit patterns, so that NaN counts as larger than every number and reaches the row's flag.
#include "qamw.h"
#include "qamw_device.hpp"
#include "qamw_w8_launch.hpp"

namespace qamw {

namespace {

constexpr int kChunk = 8;            // columns of a chunk
constexpr int kMaxWaves = 16;
constexpr float kZeroRow = 0x1p-119f;   // rows below this are zero rows: 127 / top stays finite

// 16 bytes at any address that the element type allows: gfx950 loads and stores wide at any alignment
struct __attribute__((packed, aligned(2))) Bytes16 {
    uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) Float8 {
    float v[8];
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const uint32_t a = __builtin_bit_cast(uint16_t, (__bf16)lo), b = __builtin_bit_cast(uint16_t, (__bf16)hi);
    return a | (b << 16);   // v_cvt_pk_bf16_f32: round to nearest even
}

// Columns j .. j + 7 of a row (zeros past d).
template <bool BF>
__device__ __forceinline__ void load_chunk(const void* x, int64_t row_off, int j, int d, float (&v)[kChunk]) {
    if constexpr (BF) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + row_off + j;
        if (j + kChunk <= d) {
            const Bytes16 b = *reinterpret_cast<const Bytes16*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(b.w[i] << 16);
                v[2 * i + 1] = __uint_as_float(b.w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = j + i < d ? bf16_bits_to_float(p[i]) : 0.0f;
        }
    } else {
        const float* p = reinterpret_cast<const float*>(x) + row_off + j;
        if (j + kChunk <= d) {
            const Float8 b = *reinterpret_cast<const Float8*>(p);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = b.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = j + i < d ? p[i] : 0.0f;
        }
    }
}

template <bool BF>
__device__ __forceinline__ void store_chunk(void* y, int64_t row_off, int j, int d, const float (&v)[kChunk]) {
    if constexpr (BF) {
        uint16_t* p = reinterpret_cast<uint16_t*>(y) + row_off + j;
        if (j + kChunk <= d) {
            Bytes16 b;
#pragma unroll
            for (int i = 0; i < 4; ++i) b.w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<Bytes16*>(p) = b;
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (j + i < d) p[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        }
    } else {
        float* p = reinterpret_cast<float*>(y) + row_off + j;
        if (j + kChunk <= d) {
            Float8 b;
#pragma unroll
            for (int i = 0; i < kChunk; ++i) b.v[i] = v[i];
            *reinterpret_cast<Float8*>(p) = b;
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (j + i < d) p[i] = v[i];
        }
    }
}

// silu(g) = g / (1 + exp(-g)).  v_exp_f32 and v_rcp_f32 are within an ulp; the rounded product
// -g log2(e) adds |g| 2^-24 of the exponential.  exp(-g) overflows to infinity below -88: -0 there.
__device__ __forceinline__ float silu(float g) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
    return g * __builtin_amdgcn_rcpf(1.0f + e);
}

enum { kPlain = 0, kGated = 1, kNorm = 2 };

template <int KIND, bool BF, int V>
__global__ __launch_bounds__(1024) void k_rows8(Rows8Args a) {
    __shared__ uint32_t s_top[2][kMaxWaves];
    __shared__ double s_sum[2][kMaxWaves];
    const int t = threadIdx.x, nt = blockDim.x, lane = t & (kWave - 1), wave = t / kWave, waves = nt / kWave;
    const int chunks = 2 * ((a.d + 15) / 16);   // the padding bytes of a row of codes belong to its chunks
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float v[V][kChunk];
        uint32_t top = 0;
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < V; ++k) load_chunk<BF>(a.x, row * a.ld_x, (t + k * nt) * kChunk, a.d, v[k]);
        if (KIND == kGated) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float g[kChunk];
                load_chunk<BF>(a.other, row * a.ld_other, (t + k * nt) * kChunk, a.d, g);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) v[k][i] *= silu(g[i]);
            }
        }
        if (KIND == kNorm) {
            if (a.other) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float r[kChunk];
                    load_chunk<BF>(a.other, row * a.ld_other, (t + k * nt) * kChunk, a.d, r);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[k][i] += r[i];
                }
            }
            if (a.sum) {
#pragma unroll
                for (int k = 0; k < V; ++k) store_chunk<BF>(a.sum, row * a.ld_sum, (t + k * nt) * kChunk, a.d, v[k]);
            }
#pragma unroll
            for (int k = 0; k < V; ++k)
#pragma unroll
                for (int i = 0; i < kChunk; ++i) sum += (double)v[k][i] * (double)v[k][i];
        }
        if (a.factor) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float f[kChunk];
                load_chunk<false>(a.factor, 0, (t + k * nt) * kChunk, a.d, f);
                if (KIND != kNorm && row == 0 && a.status) {
                    bool bad = false;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) bad |= (t + k * nt) * kChunk + i < a.d && !(f[i] > 0.0f);
                    if (bad) atomicOr(a.status, QAMW_FLAG_BAD_SCALE);
                }
#pragma unroll
                for (int i = 0; i < kChunk; ++i) v[k][i] *= f[i];
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                const uint32_t m = __float_as_uint(v[k][i]) & 0x7FFFFFFFu;
                top = m > top ? m : top;
            }
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) {
            const uint32_t o = __shfl_xor(top, off);
            top = o > top ? o : top;
            if (KIND == kNorm) sum += __shfl_xor(sum, off);
        }
        if (waves > 1) {
            // two buffers by turns: a wave may be one row ahead of the slowest, never two
            if (lane == 0) {
                s_top[buf][wave] = top;
                if (KIND == kNorm) s_sum[buf][wave] = sum;
            }
            __syncthreads();
            top = s_top[buf][0];
            sum = KIND == kNorm ? s_sum[buf][0] : 0.0;
            for (int w = 1; w < waves; ++w) {
                top = s_top[buf][w] > top ? s_top[buf][w] : top;
                if (KIND == kNorm) sum += s_sum[buf][w];
            }
        }
        const float ftop = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u;
        const bool zero = bad || ftop < kZeroRow;
        const float back = zero ? 0.0f : 127.0f / ftop;
        if (t == 0) {
            float s;
            if (KIND == kNorm)
                s = zero ? 0.0f : (float)((double)ftop / (127.0 * sqrt(sum / (double)a.d + a.eps)));
            else
                s = zero ? 0.0f : ftop / 127.0f;
            a.row_scale[row] = bad ? __uint_as_float(0x7FC00000u) : s;
            if (bad && a.status) atomicOr(a.status, QAMW_FLAG_NONFINITE);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = t + k * nt;
            if (c >= chunks) continue;
            uint32_t b[2] = {0, 0};
            if (!zero) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    b[i / 4] |= ((uint32_t)(int)__builtin_rintf(v[k][i] * back) & 0xFFu) << (8 * (i % 4));
            }
            *reinterpret_cast<uint2*>(a.q + row * a.ld_q + c * kChunk) = make_uint2(b[0], b[1]);
        }
    }
}

template <int KIND, bool BF>
hipError_t launch_rows(const Rows8Args& a, hipStream_t st) {
    const int chunks = 2 * ((a.d + 15) / 16);
    // chunks a thread: as few as 16 wavefronts allow
    int v = 1;
    while (v < 4 && (chunks + v - 1) / v > kMaxWaves * kWave) v *= 2;
    const int waves = ((chunks + v - 1) / v + kWave - 1) / kWave;
    const dim3 grid(a.rows < (1 << 20) ? a.rows : (1 << 20)), block(waves * kWave);
    if (v == 1)
        hipLaunchKernelGGL((k_rows8<KIND, BF, 1>), grid, block, 0, st, a);
    else if (v == 2)
        hipLaunchKernelGGL((k_rows8<KIND, BF, 2>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((k_rows8<KIND, BF, 4>), grid, block, 0, st, a);
    return hipGetLastError();
}

// 16 codes a thread; a workgroup covers tx chunks of 16 columns of 256 / tx rows, and keeps the
// reciprocals of its columns' channel scales over its rows.
template <bool BF>
__global__ __launch_bounds__(256) void k_dequant8(Dequant8Args a, int tx) {
    const int c = blockIdx.x * tx + threadIdx.x % tx;
    const int ty = 256 / tx;
    const int j = c * 16;
    if (j >= a.d) return;
    float rec[2][kChunk];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (a.scale) {
            load_chunk<false>(a.scale, 0, j + h * kChunk, a.d, rec[h]);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) rec[h][i] = j + h * kChunk + i < a.d ? 1.0f / rec[h][i] : 0.0f;
        }
    }
    for (int64_t row = (int64_t)blockIdx.y * ty + threadIdx.x / tx; row < a.rows; row += (int64_t)gridDim.y * ty) {
        const uint4 q = *reinterpret_cast<const uint4*>(a.q + row * a.ld_q + j);
        const float s = a.row_scale[row];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                v[i] = (float)(int8_t)(w[2 * h + i / 4] >> (8 * (i % 4))) * s;
                if (a.scale) v[i] *= rec[h][i];
            }
            store_chunk<BF>(a.out, row * a.ld_out, j + h * kChunk, a.d, v);
        }
    }
}

}  // namespace

hipError_t launch_quant8(const Rows8Args& a, hipStream_t st) {
    if (a.other) return a.x_bf16 ? launch_rows<kGated, true>(a, st) : launch_rows<kGated, false>(a, st);
    return a.x_bf16 ? launch_rows<kPlain, true>(a, st) : launch_rows<kPlain, false>(a, st);
}

hipError_t launch_rmsnorm8(const Rows8Args& a, hipStream_t st) {
    return a.x_bf16 ? launch_rows<kNorm, true>(a, st) : launch_rows<kNorm, false>(a, st);
}

hipError_t launch_dequant8(const Dequant8Args& a, hipStream_t st) {
    const int chunks = (a.d + 15) / 16;
    int tx = 1;
    while (tx < 256 && tx < chunks) tx *= 2;
    const int64_t rows_wg = 256 / tx, tiles = (a.rows + rows_wg - 1) / rows_wg;
    const dim3 grid((chunks + tx - 1) / tx, (unsigned)(tiles < 32768 ? tiles : 32768));
    if (a.out_bf16)
        hipLaunchKernelGGL((k_dequant8<true>), grid, dim3(256), 0, st, a, tx);
    else
        hipLaunchKernelGGL((k_dequant8<false>), grid, dim3(256), 0, st, a, tx);
    return hipGetLastError();
}

}  // namespace qamw
