// Rows of a matrix as 4-bit codes with a power of two for every 32 columns (quant4, rmsnorm4), and back
// (dequant4).
//
// A lane has 8 consecutive columns (a chunk), four lanes have a block: its largest magnitude takes two exchanges
// within the four.  The power of two comes from the exponent bits of that magnitude, so dividing by it is
// exact and v_cvt_scalef32_pk_fp4_f32 (ties to the even code, saturating) gives the codes of the exact
// quotients.  Nothing of a row is needed for a block: quant4 streams, each lane over rows of the same columns;
// rmsnorm4 holds a row in the registers of 1 to 16 wavefronts, for its sum of squares.
//
// Bound by HBM.  Measured (bytes of the rows, codes and scales, against 4.7 TB/s of a large copy): weights with channel
// scale, 13824 x 5120 bf16, 42 us (4.3 TB/s); gated 2048 x 13824 bf16, 30 us (4.3 TB/s; 40 with every value in fp64);
// norm with residual, 4096 x 5120 bf16, 28.8 us (4.8 TB/s; 41.5 with 2 chunks a thread and the weights read again for
// every row); dequant4 of 13824 x 5120 with channel scale 31 us (5.8 TB/s, part of the codes still in cache).  A single
// row takes 2.0 to 3.4 us, most of it the launch.  A group's 8 scale bytes of a row are a store of their own; rows one
// behind the other are one workgroup's, so that L2 joins them to lines (37.9 MB written for 37.6 MB of codes and
// scales).
//
// Rounding.  Values are fp32 from the load on, and every rounding is one that include/qamw_mx4.h names; the sum of squares
// and the norm's factor are fp64 up to the one rounding of the factor.  The order of the sum, which goes by the number of
// rows (norm_shape), decides that rounding only where the factor is within about d 2^-53 of the middle of two fp32 numbers.

#include <type_traits>

#include "qamw.h"
#include "qamw_device.hpp"
#include "qamw_mx4_launch.hpp"
#include "qamw_rows.hpp"

namespace qamw {

namespace {

constexpr int kMaxWaves = 16;
constexpr int kGroupChunks = kGroupCols / kChunk;
constexpr float kZeroBlock = 0x1p-119f;   // blocks below this are zero blocks: every power of two used is normal

// Lane l's value from the lane that control C names, within rows of 16 lanes.
template <int C>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, C, 0xF, 0xF, true);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E;   // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int kRor4 = 0x124, kRor8 = 0x128;   // row_ror

// A chunk of a block as codes: its 4 bytes, and in `scale` the block's byte.  The four lanes of the block call this
// together.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[kChunk], uint32_t& scale, bool& bad) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) top = top_of(top, v[i]);
    top = top_of(top, __uint_as_float(dpp<kSwap1>(__float_as_uint(top))));
    top = top_of(top, __uint_as_float(dpp<kSwap2>(__float_as_uint(top))));
    bad = !(top < __builtin_inff());
    const bool zero = bad || top < kZeroBlock;
    // top = m 2^x with 1 <= m < 2: the exponent is x - 2 up to m = 1.75 and x - 1 above
    const uint32_t byte = ((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 2;
    scale = bad ? 255u : zero ? 0u : byte;
    const float unit = __uint_as_float(byte << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], unit, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], unit, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], unit, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], unit, 3);
    return zero ? 0u : q;
}

// Writes chunk c of a row and, of 16 lanes (chunks c & -16 .. c | 15), one the four scale bytes.
__device__ __forceinline__ void store_codes(const Rows4Args& a, int64_t row, int c, uint32_t q, uint32_t scale) {
    asm volatile("" : "+v"(c));   // addresses are formed here, not kept for every chunk of a thread
    *reinterpret_cast<uint32_t*>(a.q + row * a.ld_q + (uint32_t)c * 4) = q;
    uint32_t s = scale << (8 * (c / 4 % 4));
    s |= dpp<kRor4>(s);
    s |= dpp<kRor8>(s);
    if (c % 16 == 0)
        *reinterpret_cast<uint32_t*>(a.e + c / kGroupChunks * a.ld_e + row * 8 + c / 16 % 2 * 4) = s;
}

// x g / (1 + exp(-g)) in fp64, rounded to fp32 once.  exp(-g) = 2^n 2^f with |f| <= 1/2, and 2^f by the polynomial of
// degree 8 through the Chebyshev nodes of that interval (within 2^-39.7 of itself).  With n held to +-1000, a
// quotient below every fp32 number stays one, and an infinite g gives an infinite or undefined product.
__device__ __forceinline__ float gated(float x, float g) {
    const double p = (double)x * (double)g, t = (double)g * -1.4426950408889634;
    const double n = __builtin_rint(t), f = t - n;
    double e = 1.3255224887502117e-06;
    e = __builtin_fma(e, f, 1.531007940254368e-05);
    e = __builtin_fma(e, f, 0.0001540345585240991);
    e = __builtin_fma(e, f, 0.0013333450567999414);
    e = __builtin_fma(e, f, 0.009618129159402628);
    e = __builtin_fma(e, f, 0.05550410941205934);
    e = __builtin_fma(e, f, 0.2402265069581299);
    e = __builtin_fma(e, f, 0.6931471805459335);
    e = __builtin_fma(e, f, 1.0);
    const double held = __builtin_fmin(__builtin_fmax(n, -1000.0), 1000.0);
    const double d = 1.0 + __builtin_ldexp(e, (int)held);
    double r = __builtin_amdgcn_rcp(d);   // within 2^-20 or better; two steps of Newton's iteration
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    return (float)(p * r);
}

// Gated values in fp32, which is twice as fast: for g >= -80 the exponential, the reciprocal and the products leave
// x silu(g) (and its product with a channel scale) within (|g| + 9) 2^-23 < 2^-16 of itself, as long as what is rounded
// on the way is a normal number (`lost` is set where it is not):
//   silu(g), |g| 2^-116 or more for g >= -80, and g / 2 next to 0: normal, or down to 2^-127 with an error of 2^-150,
//   where g is.  A bf16 g that is not has 7 bits or fewer, and half of it is exact.
//   x silu(g): without a scale, one below the normal numbers has code 0, or is in a zero block, whichever way it is
//   rounded, and so it is with a scale of up to kScaleLarge (2^-126 kScaleLarge is less than 0.25 in a block whose
//   largest value is kZeroBlock).  A larger scale makes a code of it (lost_before_scale).
constexpr float kGateError = 0x1p-16f, kGateLeast = -80.0f, kScaleLarge = 4.0f;
constexpr int kSubnormal = 0x90, kZero = 0x60;   // classes of v_cmp_class_f32, of both signs
template <bool BF>
__device__ __forceinline__ float gated_about(float x, float g, bool& lost) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
    if constexpr (!BF) lost |= __builtin_amdgcn_classf(g, kSubnormal);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * x;
}
__device__ __forceinline__ bool lost_before_scale(float about, float x, float g) {   // (a zero of x or g is exact)
    return __builtin_amdgcn_classf(about, kSubnormal | kZero) & (__builtin_fminf(__builtin_fabsf(x), __builtin_fabsf(g)) > 0.0f);
}

// codes_of for values that are known to within kGateError: rounding is monotone, so where both ends of every value's
// range give the same codes, and both ends of the largest one's the same power of two, those are the exact value's.
// False where they do not (of 512 values of a normal distribution in 1 wavefront of 30), and for values that are not
// finite or nearly not.
__device__ __forceinline__ bool codes_about(const float (&v)[kChunk], uint32_t& q, uint32_t& scale) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) top = top_of(top, v[i]);
    top = top_of(top, __uint_as_float(dpp<kSwap1>(__float_as_uint(top))));
    top = top_of(top, __uint_as_float(dpp<kSwap2>(__float_as_uint(top))));
    const float most = top * (1.0f + kGateError), least = top * (1.0f - kGateError);
    const uint32_t byte = ((__float_as_uint(most) + 0x1FFFFFu) >> 23) - 2;
    const bool zero = most < kZeroBlock;
    scale = zero ? 0u : byte;
    const float unit = __uint_as_float(byte << 23);
    uint32_t lo = 0, hi = 0;
    auto put = [&](uint32_t& to, float a, float b, auto at) {
        to = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(to, a, b, unit, at);
    };
    float l[kChunk], h[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) l[i] = v[i] * (1.0f - kGateError), h[i] = v[i] * (1.0f + kGateError);
    put(lo, l[0], l[1], std::integral_constant<int, 0>{});
    put(lo, l[2], l[3], std::integral_constant<int, 1>{});
    put(lo, l[4], l[5], std::integral_constant<int, 2>{});
    put(lo, l[6], l[7], std::integral_constant<int, 3>{});
    put(hi, h[0], h[1], std::integral_constant<int, 0>{});
    put(hi, h[2], h[3], std::integral_constant<int, 1>{});
    put(hi, h[4], h[5], std::integral_constant<int, 2>{});
    put(hi, h[6], h[7], std::integral_constant<int, 3>{});
    q = zero ? 0u : lo;
    return top < 0x1p127f && byte == ((__float_as_uint(least) + 0x1FFFFFu) >> 23) - 2 && (zero || (least >= kZeroBlock && lo == hi));
}

// 8 columns a thread; a workgroup covers tx chunks of rows_wg rows, 256 / tx at a time, and keeps the channel
// scales of its columns over its rows.
template <bool BF, bool GATE, bool SCALE>
__global__ __launch_bounds__(256) void k_quant4(Rows4Args a, int tx, int rows_wg) {
    const int c = blockIdx.x * tx + threadIdx.x % tx, ty = 256 / tx, j = c * kChunk;
    // (tx and the chunks of a row are multiples of 32: the lanes of a block, and the 16 of a store, leave together)
    if (c >= (a.d + kGroupCols - 1) / kGroupCols * kGroupChunks) return;
    const int have = a.d - j;   // columns of the chunk: below 8 in the last one, none behind it
    float f[kChunk];
    bool large = false;   // gated: a channel scale that makes codes of values below the normal numbers
    if constexpr (SCALE) {
        if (have >= kChunk)
            unpack<false>(*reinterpret_cast<const Float8*>(a.factor + j), f);
        else
            load_part<false>(a.factor + j, have, f);
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) bad |= i < have && !(f[i] > 0.0f);
        if (bad && blockIdx.y == 0 && a.status) atomicOr(a.status, QAMW_FLAG_BAD_SCALE);
        if constexpr (GATE) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) large |= !(__builtin_fabsf(f[i]) <= kScaleLarge);
            large = __any(large);
        }
    }
    const int64_t first = (int64_t)blockIdx.y * rows_wg, end = first + rows_wg < a.rows ? first + rows_wg : a.rows;
    bool flag = false;
    auto write = [&](int64_t row, float (&v)[kChunk], const float (&g)[kChunk]) {
        uint32_t q, s;
        if constexpr (GATE) {
            float about[kChunk], least = g[0];
            bool lost = false;
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                about[i] = gated_about<BF>(v[i], g[i], lost);
                least = __builtin_fminf(least, g[i]);
            }
            if constexpr (SCALE) {
                if (large) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) lost |= lost_before_scale(about[i], v[i], g[i]);
                }
#pragma unroll
                for (int i = 0; i < kChunk; ++i) about[i] *= f[i];
            }
            const bool sure = codes_about(about, q, s) && least >= kGateLeast && !lost;
            if (!__any(!sure)) {
                store_codes(a, row, c, q, s);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            if constexpr (GATE) v[i] = gated(v[i], g[i]);
            if constexpr (SCALE) v[i] *= f[i];
        }
        bool bad;
        q = codes_of(v, s, bad);
        flag |= bad;
        store_codes(a, row, c, q, s);
    };
    // The lanes of a block, and the 16 of a store, exchange values: whatever a lane has of the row, it comes to `write`
    // with the others.  One without a whole chunk loads the last whole one instead, and then what it has.
    const int whole = a.d / kChunk, at_j = (c < whole ? c : whole > 0 ? whole - 1 : 0) * kChunk;
    auto load = [&](int64_t row, Raw<BF>& x, Raw<BF>& o) {
        x = *reinterpret_cast<const Raw<BF>*>(at<BF>(a.x, row * a.ld_x + at_j));
        if constexpr (GATE) o = *reinterpret_cast<const Raw<BF>*>(at<BF>(a.other, row * a.ld_other + at_j));
    };
    auto take = [&](int64_t row, const Raw<BF>& x, const Raw<BF>& o) {
        float v[kChunk], g[kChunk];
        unpack<BF>(x, v);
        if constexpr (GATE) unpack<BF>(o, g);
        if (have < kChunk) {
            load_part<BF>(at<BF>(a.x, row * a.ld_x + j), have, v);
            if constexpr (GATE) load_part<BF>(at<BF>(a.other, row * a.ld_other + j), have, g);
        }
        write(row, v, g);
    };
    int64_t row = first + threadIdx.x / tx;
    if (whole > 0) {
        // four rows at a time, every load under way before the first is used
        constexpr int U = 4;
        for (; row + (U - 1) * ty < end; row += U * ty) {
            Raw<BF> x[U], o[U];
#pragma unroll
            for (int u = 0; u < U; ++u) load(row + u * ty, x[u], o[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) take(row + u * ty, x[u], o[u]);
        }
    }
    for (; row < end; row += ty) {
        Raw<BF> x{}, o{};
        if (whole > 0) load(row, x, o);
        take(row, x, o);
    }
    if (flag && a.status) atomicOr(a.status, QAMW_FLAG_NONFINITE);
}

// Threads across a row: a power of two from 32 to 256 that leaves few of them without a chunk.
int across(int chunks) {
    int tx = 32;
    for (int wide = 64; wide <= 256; wide *= 2)
        if ((chunks + wide - 1) / wide * wide <= (chunks + tx - 1) / tx * tx) tx = wide;
    return tx;
}

template <bool BF, bool GATE, bool SCALE>
hipError_t launch_quant(const Rows4Args& a, hipStream_t st) {
    const int chunks = (a.d + kGroupCols - 1) / kGroupCols * kGroupChunks, tx = across(chunks), ty = 256 / tx;
    const int64_t cols = (chunks + tx - 1) / tx, most = (2048 + cols - 1) / cols;   // 8 workgroups a compute unit
    int64_t rows_wg = (a.rows + most - 1) / most;
    rows_wg = (rows_wg + ty - 1) / ty * ty;
    if (rows_wg > 16) rows_wg = (rows_wg + 15) / 16 * 16;   // whole lines of scales
    const dim3 grid((unsigned)cols, (unsigned)((a.rows + rows_wg - 1) / rows_wg));
    return launch_kernel(k_quant4<BF, GATE, SCALE>, grid, 256, 0, st, a, tx, (int)rows_wg);
}

template <bool BF>
hipError_t launch_quant(const Rows4Args& a, hipStream_t st) {
    if (a.other) return a.factor ? launch_quant<BF, true, true>(a, st) : launch_quant<BF, true, false>(a, st);
    return a.factor ? launch_quant<BF, false, true>(a, st) : launch_quant<BF, false, false>(a, st);
}

// Wavefronts of a workgroup, and with them registers of a lane, by the registers that v chunks need.
constexpr int max_waves(int v) { return v <= 2 ? 16 : v <= 4 ? 12 : 8; }

// row_waves wavefronts a row: one row a workgroup, or, with one wavefront a row, blockDim / 64.  Chunk t + k threads
// of the row's whole groups is thread t's; a thread without one at some k loads the last one again, so that every load
// is unconditional.  A part of a group at the end is the first 32 threads', a chunk each.
template <bool BF, bool FACTOR, int V>
__global__ __launch_bounds__(max_waves(V) * kWave) void k_rmsnorm4(Rows4Args a, int row_waves, int keep) {
    // FACTOR: a thread's factors, kept over its rows (with `keep`: as long as they fit)
    extern __shared__ __align__(16) float4 s_factor[];
    bool kept = false;
    __shared__ double s_sum[2][kMaxWaves];
    // (in scalar registers: a row's addresses are then a scalar base and an offset of 32 bits)
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int rows_wg = blockDim.x / kWave / row_waves, part = wave % row_waves;
    const int t = part * kWave + lane, nt = row_waves * kWave;
    const int chunks = a.d / kGroupCols * kGroupChunks, end_c = chunks + t, have = a.d - end_c * kChunk;
    const bool end = a.d % kGroupCols && t < kGroupChunks;
    int chunk[V];
#pragma unroll
    for (int k = 0; k < V; ++k) chunk[k] = t + k * nt < chunks ? t + k * nt : chunks - 1;
    bool flag = false;
    int buf = 0;
    for (int64_t row = (int64_t)blockIdx.x * rows_wg + wave / row_waves; row < a.rows;
         row += (int64_t)gridDim.x * rows_wg, buf ^= 1) {
        const void* x = at<BF>(a.x, row * a.ld_x);
        const void* other = at<BF>(a.other, row * a.ld_other);
        void* sum_out = const_cast<void*>(at<BF>(a.sum, row * a.ld_sum));
        float v[V][kChunk], last[kChunk];
        double sum = 0.0;
        if (chunks > 0) {
            Raw<BF> rx[V], ro[V];
#pragma unroll
            for (int k = 0; k < V; ++k) rx[k] = *reinterpret_cast<const Raw<BF>*>(at<BF>(x, chunk[k] * kChunk));
            if (a.other) {
#pragma unroll
                for (int k = 0; k < V; ++k) ro[k] = *reinterpret_cast<const Raw<BF>*>(at<BF>(other, chunk[k] * kChunk));
            }
#pragma unroll
            for (int k = 0; k < V; ++k) unpack<BF>(rx[k], v[k]);
            if (a.other) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float o[kChunk];
                    unpack<BF>(ro[k], o);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[k][i] += o[i];
                }
            }
            if (a.sum) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (t + k * nt < chunks) store_chunk<BF>(const_cast<void*>(at<BF>(sum_out, chunk[k] * kChunk)), v[k]);
            }
            // (a chunk loaded again does not count: with h in place of x, its thread may have written it already)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                double q = 0.0;
#pragma unroll
                for (int i = 0; i < kChunk; ++i) q = __builtin_fma((double)v[k][i], (double)v[k][i], q);
                sum += t + k * nt < chunks ? q : 0.0;
            }
        }
        if (end) {
            load_part<BF>(at<BF>(x, end_c * kChunk), have, last);
            if (a.other) {
                float o[kChunk];
                load_part<BF>(at<BF>(other, end_c * kChunk), have, o);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) last[i] += o[i];
            }
            if (a.sum) store_part<BF>(const_cast<void*>(at<BF>(sum_out, end_c * kChunk)), have, last);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) sum = __builtin_fma((double)last[i], (double)last[i], sum);
        }
        if constexpr (FACTOR) {
            if (chunks > 0) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    Float8 f;
                    float4* mine = s_factor + 2 * k * nt + t;   // wavefronts of other rows write the same there
                    asm volatile("" ::: "memory");   // a chunk's factors at a time: together they need scratch memory
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
                    for (int i = 0; i < kChunk; ++i) v[k][i] *= f.v[i];
                }
                kept = keep;
            }
            if (end) {
                float f[kChunk];
                load_part<false>(a.factor + end_c * kChunk, have, f);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) last[i] *= f[i];
            }
        }
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
        if (row_waves > 1) {   // then the workgroup has one row
            // two buffers by turns: a wave may be one row ahead of the slowest, never two
            if (lane == 0) s_sum[buf][wave] = sum;
            __syncthreads();
            sum = s_sum[buf][0];
            for (int w = 1; w < row_waves; ++w) sum += s_sum[buf][w];
        }
        const float f = (float)(1.0 / sqrt(sum / (double)a.d + a.eps));
        if (chunks > 0) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                asm volatile("" ::: "memory");
#pragma unroll
                for (int i = 0; i < kChunk; ++i) v[k][i] *= f;
                uint32_t s;
                bool bad;
                const uint32_t q = codes_of(v[k], s, bad);
                if (t + k * nt < chunks) {   // (of 32 lanes all or none)
                    flag |= bad;
                    store_codes(a, row, chunk[k], q, s);
                }
            }
        }
        if (end) {
            // behind the row: zeros, whatever the factor is
#pragma unroll
            for (int i = 0; i < kChunk; ++i) last[i] = i < have ? last[i] * f : 0.0f;
            uint32_t s;
            bool bad;
            const uint32_t q = codes_of(last, s, bad);
            flag |= bad;
            store_codes(a, row, end_c, q, s);
        }
    }
    if (flag && a.status) atomicOr(a.status, QAMW_FLAG_NONFINITE);
}

// How a row is spread: v chunks a thread, w wavefronts.  Many rows fill the chip by themselves, and a thread has 4 chunks,
// so that a compute unit has many bytes under way and few wavefronts wait for each other (4096 x 5120 bf16 with a
// residual: 1 chunk 43.6 us, 2: 33.2, 4: 31.3, 5: 31.6, 8: 37.9); fewer values than 4.5 million are spread over more
// wavefronts (512 x 4096: 2 chunks 5.3 us, 4: 6.3; 1024 x 5120: 10.4 and 9.8; one row of 4096: 3.5 and 4.3).
struct NormShape {
    int v, w;
};
NormShape norm_shape(int rows, int d) {
    const int chunks = d / kGroupCols * kGroupChunks, waves = chunks < kWave ? 1 : (chunks + kWave - 1) / kWave;
    if (waves == 1) return {1, 1};
    for (const int v : {2, 4})
        if ((v == 4 || (int64_t)rows * d < 4500000) && (waves + v - 1) / v <= max_waves(v)) return {v, (waves + v - 1) / v};
    return {8, (waves + 7) / 8};   // up to 32768 columns
}

template <bool BF, bool FACTOR, int V>
hipError_t launch_norm(const Rows4Args& a, int w, hipStream_t st) {
    const int rows_wg = w == 1 ? 4 : 1;
    // the factors of a row: in LDS from the first row of a workgroup on, and then a workgroup has many rows
    // (about as many workgroups as fit at once)
    const size_t bytes = FACTOR ? (size_t)V * 32 * w * kWave : 0;
    const bool keep = bytes > 0 && bytes <= 65536;
    int64_t wgs = ((int64_t)a.rows + rows_wg - 1) / rows_wg;
    const int64_t most = keep ? 256 * (12 / (rows_wg * w) > 0 ? 12 / (rows_wg * w) : 1) : 1 << 20;
    wgs = wgs < most ? wgs : most;
    return launch_kernel(k_rmsnorm4<BF, FACTOR, V>, dim3((unsigned)wgs), rows_wg * w * kWave, keep ? bytes : 0, st, a, w,
                         keep ? 1 : 0);
}

template <bool BF, bool FACTOR>
hipError_t launch_norm(const Rows4Args& a, hipStream_t st) {
    const NormShape s = norm_shape(a.rows, a.d);
    switch (s.v) {
    case 1: return launch_norm<BF, FACTOR, 1>(a, s.w, st);
    case 2: return launch_norm<BF, FACTOR, 2>(a, s.w, st);
    case 4: return launch_norm<BF, FACTOR, 4>(a, s.w, st);
    default: return launch_norm<BF, FACTOR, 8>(a, s.w, st);
    }
}

// 8 codes a thread; a workgroup covers tx chunks of rows_wg rows, 256 / tx at a time, and keeps the reciprocals of its
// columns' channel scales over its rows.
template <bool BF, bool SCALE>
__global__ __launch_bounds__(256) void k_dequant4(Dequant4Args a, int tx, int rows_wg) {
    const int c = blockIdx.x * tx + threadIdx.x % tx, ty = 256 / tx, j = c * kChunk, have = a.d - j;
    if (have <= 0) return;
    float rec[kChunk];
    if constexpr (SCALE) {
        if (have >= kChunk)
            unpack<false>(*reinterpret_cast<const Float8*>(a.scale + j), rec);
        else
            load_part<false>(a.scale + j, have, rec);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) rec[i] = 1.0f / rec[i];
    }
    const int64_t first = (int64_t)blockIdx.y * rows_wg, end = first + rows_wg < a.rows ? first + rows_wg : a.rows;
    const uint8_t* e = a.e + c / kGroupChunks * a.ld_e + c / 4 % 8;
    auto write = [&](int64_t row, uint32_t q, uint32_t byte) {
        // 2^-127 is no normal number; 255 is NaN
        const float unit = __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3)};
        float v[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            v[i] = p[i / 2][i % 2] * unit;
            if constexpr (SCALE) v[i] *= rec[i];
        }
        void* y = const_cast<void*>(at<BF>(a.out, row * a.ld_out + j));
        if (have >= kChunk)
            store_chunk<BF>(y, v);
        else
            store_part<BF>(y, have, v);
    };
    int64_t row = first + threadIdx.x / tx;
    // four rows at a time, every load under way before the first is used
    constexpr int U = 4;
    for (; row + (U - 1) * ty < end; row += U * ty) {
        uint32_t q[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            q[u] = *reinterpret_cast<const uint32_t*>(a.q + (row + u * ty) * a.ld_q + c * 4);
            s[u] = e[(row + u * ty) * 8];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) write(row + u * ty, q[u], s[u]);
    }
    for (; row < end; row += ty)
        write(row, *reinterpret_cast<const uint32_t*>(a.q + row * a.ld_q + c * 4), e[row * 8]);
}

template <bool BF, bool SCALE>
hipError_t launch_dequant(const Dequant4Args& a, hipStream_t st) {
    const int chunks = (a.d + kChunk - 1) / kChunk, tx = across(chunks), ty = 256 / tx;
    const int64_t cols = (chunks + tx - 1) / tx, most = (2048 + cols - 1) / cols;   // 8 workgroups a compute unit
    int64_t rows_wg = (a.rows + most - 1) / most;
    rows_wg = (rows_wg + ty - 1) / ty * ty;
    const dim3 grid((unsigned)cols, (unsigned)((a.rows + rows_wg - 1) / rows_wg));
    return launch_kernel(k_dequant4<BF, SCALE>, grid, 256, 0, st, a, tx, (int)rows_wg);
}

}  // namespace

hipError_t launch_quant4(const Rows4Args& a, hipStream_t st) {
    return a.x_bf16 ? launch_quant<true>(a, st) : launch_quant<false>(a, st);
}

hipError_t launch_rmsnorm4(const Rows4Args& a, hipStream_t st) {
    if (a.x_bf16) return a.factor ? launch_norm<true, true>(a, st) : launch_norm<true, false>(a, st);
    return a.factor ? launch_norm<false, true>(a, st) : launch_norm<false, false>(a, st);
}

hipError_t launch_dequant4(const Dequant4Args& a, hipStream_t st) {
    if (a.scale) return a.out_bf16 ? launch_dequant<true, true>(a, st) : launch_dequant<false, true>(a, st);
    return a.out_bf16 ? launch_dequant<true, false>(a, st) : launch_dequant<false, false>(a, st);
}

}  // namespace qamw
