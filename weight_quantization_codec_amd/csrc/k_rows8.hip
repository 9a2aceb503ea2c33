// Rows of a matrix as 8-bit codes with a scale each (quant8, rmsnorm8), and back (dequant8).
//
// k_rows8: a row in the registers of 1 to 16 wavefronts: every thread holds V chunks of 8 consecutive
// columns, chunk t + v * threads, so a wavefront's loads are contiguous.  One pass over HBM: the row's
// largest magnitude (and for the norm its sum of squares) is reduced over the row's wavefronts, then the
// codes are formed from the registers.  The norm's factor 1 / rms is the same for the whole row, so it
// changes the row scale and no code: codes need the largest magnitude only, and both reductions share one
// barrier.
//
// Bound by HBM.  Measured (bytes of the rows and codes, against 5.1 TB/s of a large copy): norm with
// residual, 4096 x 5120 bf16, 28.6 us (5.1 TB/s); weights with channel scale, 13824 x 5120 bf16, 47 us
// (4.5 TB/s; 54 with the scales read again for every row, 42 without a scale); gated 2048 x 13824 bf16, 31 us
// (4.6 TB/s); dequant8 of 13824 x 5120 with channel scale 37 us (5.7 TB/s, part of the codes still in cache; 46.6 us
// from memory; to fp32 147 us, 2.4 TB/s).
// A single row takes 2.7 to 3.4 us, most of it the launch.
//
// Rounding.  Values are fp32 from the load on; the sum of squares is fp64, which holds the square of
// every fp32 value and adds 32768 of them without overflow or loss that matters.  NaN counts as larger
// than every number in the row's maximum, and so reaches the row's flag.
#include <type_traits>

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

// The 8 columns of a chunk as they are stored, at any alignment of the elements.
template <bool BF>
using Raw = std::conditional_t<BF, Bytes16, Float8>;

template <bool BF>
__device__ __forceinline__ const void* at(const void* p, int64_t element) {
    return reinterpret_cast<const char*>(p) + element * (BF ? 2 : 4);
}

template <bool BF>
__device__ __forceinline__ void unpack(const Raw<BF>& b, float (&v)[kChunk]) {
    if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(b.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(b.w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = b.v[i];
    }
}

// The first n < 8 columns of a chunk, and zeros.
template <bool BF>
__device__ __forceinline__ void load_part(const void* p, int n, float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        v[i] = 0.0f;
        if (i < n) {
            if constexpr (BF)
                v[i] = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]);
            else
                v[i] = reinterpret_cast<const float*>(p)[i];
        }
    }
}

template <bool BF>
__device__ __forceinline__ void store_chunk(void* y, const float (&v)[kChunk]) {
    if constexpr (BF) {
        Bytes16 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) b.w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<Bytes16*>(y) = b;
    } else {
        Float8 b;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) b.v[i] = v[i];
        *reinterpret_cast<Float8*>(y) = b;
    }
}

template <bool BF>
__device__ __forceinline__ void store_part(void* y, int n, const float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
        if (i < n) {
            if constexpr (BF)
                reinterpret_cast<uint16_t*>(y)[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
            else
                reinterpret_cast<float*>(y)[i] = v[i];
        }
}

// silu(g) = g / (1 + exp(-g)).  v_exp_f32 and v_rcp_f32 are within an ulp; the rounded product
// -g log2(e) adds |g| 2^-24 of the exponential.  exp(-g) overflows to infinity below -88: -0 there.
__device__ __forceinline__ float silu(float g) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
    return g * __builtin_amdgcn_rcpf(1.0f + e);
}

enum { kPlain = 0, kGated = 1, kNorm = 2 };

// The larger of a magnitude and |v|; NaN if either is (v_maximum3_f32).
__device__ __forceinline__ float top_of(float top, float v) {
    return __builtin_elementwise_maximum(top, __builtin_fabsf(v));
}

// Codes of 8 values: fl32(v back) is at most 127; adding 1.5 2^23 rounds it to the nearest whole number,
// ties to even, and leaves that as two's complement in the low bits.
__device__ __forceinline__ uint2 codes_of(const float (&v)[kChunk], float back) {
    uint32_t q[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) q[i] = __float_as_uint(v[i] * back + 12582912.0f);
    uint32_t b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400u) |
               __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x04000C0Cu);
    return make_uint2(b[0], b[1]);
}

// Wavefronts of a workgroup, and with them registers of a lane, by the registers that v chunks need.
constexpr int max_waves(int v) { return v <= 2 ? 16 : v <= 5 ? 12 : 8; }

// row_waves wavefronts a row: one row a workgroup, or, with one wavefront a row, blockDim / 64.
template <int KIND, bool BF, bool FACTOR, int V>
__global__ __launch_bounds__(max_waves(V) * kWave) void k_rows8(Rows8Args a, int row_waves, int keep) {
    // FACTOR: a thread's factors, kept over its rows (with `keep`: as long as they fit)
    extern __shared__ __align__(16) float4 s_factor[];
    bool kept = false;
    __shared__ float s_top[2][kMaxWaves];
    __shared__ double s_sum[2][kMaxWaves];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int rows_wg = blockDim.x / kWave / row_waves, part = wave % row_waves;
    const int t = part * kWave + lane, nt = row_waves * kWave;
    // Whole chunks.  A thread without one at some k loads the last one again: every load is unconditional,
    // so all of them are under way at once (with a branch for each, a row took twice as long).
    const int full = a.d / kChunk, rest = a.d % kChunk, chunks = 2 * ((a.d + 15) / 16);
    int chunk[V];
#pragma unroll
    for (int k = 0; k < V; ++k) chunk[k] = t + k * nt < full ? t + k * nt : full - 1;
    int buf = 0;
    for (int64_t row = (int64_t)blockIdx.x * rows_wg + wave / row_waves; row < a.rows;
         row += (int64_t)gridDim.x * rows_wg, buf ^= 1) {
        const void* x = at<BF>(a.x, row * a.ld_x);
        const void* other = at<BF>(a.other, row * a.ld_other);
        void* sum_out = const_cast<void*>(at<BF>(a.sum, row * a.ld_sum));
        float v[V][kChunk], last[kChunk];   // `last`: the columns behind the whole chunks, thread 0's
        float top = 0.0f;
        double sum = 0.0;
        if (full > 0) {
            Raw<BF> rx[V], ro[V];
#pragma unroll
            for (int k = 0; k < V; ++k) rx[k] = *reinterpret_cast<const Raw<BF>*>(at<BF>(x, chunk[k] * kChunk));
            if (KIND != kPlain && a.other) {
#pragma unroll
                for (int k = 0; k < V; ++k) ro[k] = *reinterpret_cast<const Raw<BF>*>(at<BF>(other, chunk[k] * kChunk));
            }
#pragma unroll
            for (int k = 0; k < V; ++k) unpack<BF>(rx[k], v[k]);
            if (KIND != kPlain && a.other) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float o[kChunk];
                    unpack<BF>(ro[k], o);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[k][i] = KIND == kGated ? v[k][i] * silu(o[i]) : v[k][i] + o[i];
                }
            }
        }
        if (rest && t == 0) {
            load_part<BF>(at<BF>(x, full * kChunk), rest, last);
            if (KIND != kPlain && a.other) {
                float o[kChunk];
                load_part<BF>(at<BF>(other, full * kChunk), rest, o);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) last[i] = KIND == kGated ? last[i] * silu(o[i]) : last[i] + o[i];
            }
        }
        if (KIND == kNorm) {
            if (a.sum) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (t + k * nt < full) store_chunk<BF>(const_cast<void*>(at<BF>(sum_out, chunk[k] * kChunk)), v[k]);
                if (rest && t == 0) store_part<BF>(const_cast<void*>(at<BF>(sum_out, full * kChunk)), rest, last);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                double s = 0.0;
#pragma unroll
                for (int i = 0; i < kChunk; ++i) s = __builtin_fma((double)v[k][i], (double)v[k][i], s);
                sum += t + k * nt < full ? s : 0.0;
            }
            if (rest && t == 0) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) sum = __builtin_fma((double)last[i], (double)last[i], sum);
            }
        }
        if constexpr (FACTOR) {
            bool bad = false;
            if (full > 0) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    Float8 f;
                    float4* mine = s_factor + 2 * k * nt + t;   // wavefronts of other rows write the same there
                    if (kept) {
                        const float4 lo = mine[0], hi = mine[nt];
                        f = {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
                    } else {
                        f = *reinterpret_cast<const Float8*>(a.factor + chunk[k] * kChunk);
                        if (keep) {
                            mine[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
                            mine[nt] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        v[k][i] *= f.v[i];
                        if (KIND != kNorm) bad |= !(f.v[i] > 0.0f);
                    }
                }
                kept = keep;
            }
            if (rest && t == 0) {
                float f[kChunk];
                load_part<false>(a.factor + full * kChunk, rest, f);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    last[i] *= f[i];
                    if (KIND != kNorm) bad |= i < rest && !(f[i] > 0.0f);
                }
            }
            if (KIND != kNorm && row == 0 && bad && a.status) atomicOr(a.status, QAMW_FLAG_BAD_SCALE);
        }
        // (a chunk loaded again does not count: with h in place of x, its thread may have written it already)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < kChunk; ++i) m = top_of(m, v[k][i]);
            top = t + k * nt < full ? top_of(top, m) : top;
        }
        if (rest && t == 0) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) top = top_of(top, last[i]);
        }
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) {
            top = top_of(top, __shfl_xor(top, off));
            if (KIND == kNorm) sum += __shfl_xor(sum, off);
        }
        if (row_waves > 1) {   // then the workgroup has one row
            // two buffers by turns: a wave may be one row ahead of the slowest, never two
            if (lane == 0) {
                s_top[buf][wave] = top;
                if (KIND == kNorm) s_sum[buf][wave] = sum;
            }
            __syncthreads();
            top = s_top[buf][0];
            sum = KIND == kNorm ? s_sum[buf][0] : 0.0;
            for (int w = 1; w < row_waves; ++w) {
                top = top_of(top, s_top[buf][w]);
                if (KIND == kNorm) sum += s_sum[buf][w];
            }
        }
        const bool bad = !(top < __builtin_inff());
        const bool zero = bad || top < kZeroRow;
        const float back = zero ? 0.0f : 127.0f / top;
        if (t == 0) {
            float s;
            if (KIND == kNorm)
                s = zero ? 0.0f : (float)((double)top / (127.0 * sqrt(sum / (double)a.d + a.eps)));
            else
                s = zero ? 0.0f : top / 127.0f;
            a.row_scale[row] = bad ? __uint_as_float(0x7FC00000u) : s;
            if (bad && a.status) atomicOr(a.status, QAMW_FLAG_NONFINITE);
        }
        int8_t* q = a.q + row * a.ld_q;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (t + k * nt < full)
                *reinterpret_cast<uint2*>(q + chunk[k] * kChunk) = zero ? make_uint2(0, 0) : codes_of(v[k], back);
        if (t == 0 && full < chunks) {   // the columns behind the whole chunks, and the row's padding
            *reinterpret_cast<uint2*>(q + full * kChunk) = !rest || zero ? make_uint2(0, 0) : codes_of(last, back);
            if (full + 1 < chunks) *reinterpret_cast<uint2*>(q + (full + 1) * kChunk) = make_uint2(0, 0);
        }
    }
}

// How a row is spread: v chunks a thread, w wavefronts.  Many rows fill the chip by themselves: of bf16 4, 5
// or 8 chunks, whichever leaves the fewest lanes idle, so that a compute unit has many bytes under way and few
// wavefronts wait for each other (13824 x 5120 bf16, 1 chunk a thread 107 us, 2: 67, 4: 58, 5: 54); of fp32,
// twice the bytes, 4 (8 chunks of fp32 do not fit the registers of 8 wavefronts, and a kernel with scratch
// memory takes 12 us longer to start: for the widest rows only).  Less work is spread over more wavefronts: 2
// chunks below 3 million values (512 x 4096 norm bf16: 2 chunks 6.1 us, 4: 6.8; 1000 x 6336: 15.3 and 12.7), 1 for
// up to 256 rows (256 x 2048: 3.8 us, 2: 4.1).  Each threshold rests on the sizes named with it, no more.
struct RowShape {
    int v, w;
};
RowShape row_shape(int rows, int d, bool bf) {
    const int full = d / kChunk, waves = full < kWave ? 1 : (full + kWave - 1) / kWave;
    RowShape best{0, 0};
    auto consider = [&](int v) {
        const int w = (waves + v - 1) / v;
        if (w <= max_waves(v) && (best.v == 0 || v * w < best.v * best.w)) best = {v, w};
    };
    if (waves == 1 || (rows <= 256 && waves <= 10)) consider(1);
    else if (waves == 2 || (int64_t)rows * d < 3000000) consider(2);
    if (best.v == 0) consider(4);
    if (best.v == 4 && bf) consider(5), consider(8);
    if (best.v == 0) consider(8);   // up to 32768 columns
    return best;
}

template <int KIND, bool BF, bool FACTOR, int V>
hipError_t launch_rows_v(const Rows8Args& a, int w, hipStream_t st) {
    const int rows_wg = w == 1 ? 4 : 1;
    // the factors of a row: in LDS from the first row of a workgroup on, and then a workgroup has many rows
    // (about as many workgroups as fit at once)
    const size_t bytes = FACTOR ? (size_t)V * 32 * w * kWave : 0;
    const bool keep = bytes > 0 && bytes <= 65536;
    int64_t wgs = ((int64_t)a.rows + rows_wg - 1) / rows_wg;
    const int64_t most = keep ? 256 * (12 / (rows_wg * w) > 0 ? 12 / (rows_wg * w) : 1) : 1 << 20;
    wgs = wgs < most ? wgs : most;
    return launch_kernel(k_rows8<KIND, BF, FACTOR, V>, dim3((unsigned)wgs), rows_wg * w * kWave, keep ? bytes : 0, st, a,
                         w, keep ? 1 : 0);
}

template <int KIND, bool BF, bool FACTOR>
hipError_t launch_rows_f(const Rows8Args& a, hipStream_t st) {
    const RowShape s = row_shape(a.rows, a.d, BF);
    switch (s.v) {
    case 1: return launch_rows_v<KIND, BF, FACTOR, 1>(a, s.w, st);
    case 2: return launch_rows_v<KIND, BF, FACTOR, 2>(a, s.w, st);
    case 4: return launch_rows_v<KIND, BF, FACTOR, 4>(a, s.w, st);
    case 5:
        if constexpr (BF) return launch_rows_v<KIND, BF, FACTOR, 5>(a, s.w, st);
        [[fallthrough]];
    default: return launch_rows_v<KIND, BF, FACTOR, 8>(a, s.w, st);
    }
}

template <int KIND, bool BF>
hipError_t launch_rows(const Rows8Args& a, hipStream_t st) {
    return a.factor ? launch_rows_f<KIND, BF, true>(a, st) : launch_rows_f<KIND, BF, false>(a, st);
}

// 16 codes a thread; a workgroup covers tx chunks of 16 columns of 256 / tx rows, and keeps the
// reciprocals of its columns' channel scales over its rows.
template <bool BF, bool SCALE>
__global__ __launch_bounds__(256) void k_dequant8(Dequant8Args a, int tx) {
    const int c = blockIdx.x * tx + threadIdx.x % tx, ty = 256 / tx, j = c * 16;
    if (j >= a.d) return;
    const int left = a.d - j;
    float rec[2][kChunk];
    if constexpr (SCALE) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = left - h * kChunk;
            if (n >= kChunk)
                unpack<false>(*reinterpret_cast<const Float8*>(a.scale + j + h * kChunk), rec[h]);
            else
                load_part<false>(a.scale + j + h * kChunk, n, rec[h]);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) rec[h][i] = 1.0f / rec[h][i];
        }
    }
    const int64_t by = (int64_t)gridDim.y * ty;
    int64_t row = (int64_t)blockIdx.y * ty + threadIdx.x / tx;
    auto read = [&](int64_t r, uint4& q, float& s) {
        q = *reinterpret_cast<const uint4*>(a.q + r * a.ld_q + j);
        s = a.row_scale[r];
    };
    auto write = [&](int64_t r, uint4 q, float s) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                v[i] = (float)(int8_t)(w[2 * h + i / 4] >> (8 * (i % 4))) * s;
                if constexpr (SCALE) v[i] *= rec[h][i];
            }
            void* y = const_cast<void*>(at<BF>(a.out, r * a.ld_out + j + h * kChunk));
            const int n = left - h * kChunk;
            if (n >= kChunk)
                store_chunk<BF>(y, v);
            else
                store_part<BF>(y, n, v);
        }
    };
    // four rows at a time, every load under way before the first is used
    for (; row + 3 * by < a.rows; row += 4 * by) {
        uint4 q[4];
        float s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) read(row + u * by, q[u], s[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) write(row + u * by, q[u], s[u]);
    }
    for (; row < a.rows; row += by) {
        uint4 q;
        float s;
        read(row, q, s);
        write(row, q, s);
    }
}

template <bool BF, bool SCALE>
hipError_t launch_dequant(const Dequant8Args& a, hipStream_t st) {
    const int chunks = (a.d + 15) / 16;
    // chunks across a workgroup: a power of two that leaves few threads without one (64 for 320 chunks)
    int tx = 1;
    while (tx < 64 && tx < chunks) tx *= 2;
    for (int wide = 2 * tx; wide <= 256 && wide / 2 < chunks; wide *= 2)
        if ((chunks + wide - 1) / wide * wide <= (chunks + tx - 1) / tx * tx) tx = wide;
    const int64_t rows_wg = 256 / tx, tiles = (a.rows + rows_wg - 1) / rows_wg;
    const int64_t cols = (chunks + tx - 1) / tx, most = (2048 + cols - 1) / cols;   // 8 workgroups a compute unit
    const dim3 grid((unsigned)cols, (unsigned)(tiles < most ? tiles : most));
    return launch_kernel(k_dequant8<BF, SCALE>, grid, 256, 0, st, a, tx);
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
    if (a.scale) return a.out_bf16 ? launch_dequant<true, true>(a, st) : launch_dequant<false, true>(a, st);
    return a.out_bf16 ? launch_dequant<true, false>(a, st) : launch_dequant<false, false>(a, st);
}

}  // namespace qamw
