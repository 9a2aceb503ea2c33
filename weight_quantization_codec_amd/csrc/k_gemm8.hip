// Product of 8-bit matrices: y[m][n] = xs_m ws_n sum_k xq[m][k] wq[n][k], exact 32-bit integer sums on
// the matrix cores (v_mfma_i32_32x32x32_i8).
//
// Both operands have their columns k contiguous.  An operand of the instruction is 16 consecutive bytes
// of one row a lane; which k a byte belongs to does not matter as long as both operands agree, so the
// rows are used as they are stored.
//
// Two kernels.  k_gemm8 forms a tile of y a workgroup, with the operands in stages of 128 bytes of k in LDS;
// where the tiles do not fill the chip, k is split over workgroups too and k_gemm8_join adds their sums.
// k_gemm8_thin, for few activation rows, spreads the weight rows evenly over the compute units and splits k
// over the wavefronts of a workgroup.  plan() (qamw_w8_plan.hpp) chooses.
#include <atomic>
#include <type_traits>

#include "qamw_device.hpp"
#include "qamw_w8_launch.hpp"
#include "qamw_w8_plan.hpp"

namespace qamw {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// f(0), .., f(N - 1) with the index a compile-time constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<N, I + 1>(f);
    }
}

// 16 bytes of output at any alignment of its elements
struct __attribute__((packed, aligned(2))) Out16 {
    uint32_t w[4];
};

struct __attribute__((packed, aligned(2))) Out8 {
    uint32_t w[2];
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const uint32_t a = __builtin_bit_cast(uint16_t, (__bf16)lo), b = __builtin_bit_cast(uint16_t, (__bf16)hi);
    return a | (b << 16);
}

// 16 bytes a lane from a buffer into LDS at lds + 16 lane (lds uniform), without registers between.
// Written as assembly: the compiler would wait for every such load before any read of LDS, while the
// kernel knows which stage a load fills and waits for that one (wait_stage).  The instruction has no
// register output; M0, which nothing else in these kernels uses, needs one wait state before it.
__device__ __forceinline__ void load_lds16(u32x4 rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory");
}

// A buffer descriptor: `size` bytes from `base` on, loads past them give zeros.
__device__ __forceinline__ u32x4 rsrc_of(uint64_t base, uint32_t size) {
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((uint32_t)base);
    r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(base >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane(size);
    r[3] = 0x00020000u;
    return r;
}

// Waits until at most N of the wavefront's loads and none of its LDS reads are under way, then for the
// workgroup.
template <int N>
__device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The same for LDS reads alone: behind it the workgroup has read what it has asked for.
__device__ __forceinline__ void wait_reads() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a tile leaves: y, or its sums over a part of k, to be joined.
enum { kF32 = 0, kBf16 = 1, kSums = 2 };
__host__ __device__ constexpr int sums_pitch(int n) { return (n + 63) / 64 * 64; }

// A tile of BM activation rows by BN weight rows, WM x 4 / WM wavefronts, S stages of KS bytes of k in LDS.
//
// What bounds it.  256 x 256 x 128 codes are 64 matrix instructions of 32 cycles for each of the 4 SIMDs, 2048
// cycles, in which LDS delivers 128 KiB to the operands and takes in 64 KiB.  On 8192 x 13824 x 5120 the loads
// alone take 375 us (of 480), with L2 delivering 12 to 13 TB/s to the compute units: the larger the tile, the
// less there is to deliver, so the tile takes all registers (a wavefront's 128 x 128 sums are 256 registers a
// lane, one wavefront a SIMD).  Matrix instructions on random codes from registers alone reach 3300 TOP/s,
// as the clock falls to 1.7 GHz.
//   step by step (us, that size): all of a refill's loads behind one sub-step 539; over 24 instructions 499;
//   the stage's last operands read early (FA = 0), so that a refill has 6 of 4 sub-steps' time until it is
//   needed, over 48 instructions 467.  64-byte stages (more of them) 540 to 570; 128 x 256 tiles, two
//   workgroups a compute unit, 630; a persistent workgroup that loads its next tile during the output 506.
template <int BM, int BN, int WM, int KS, int S, int SP, int FA>
struct TileCfg {
    static constexpr int kWN = 4 / WM, kRowsM = BM / WM, kRowsN = BN / kWN;   // a wavefront's part
    static constexpr int kTM = kRowsM / 32, kTN = kRowsN / 32;                // in blocks of 32 x 32
    static constexpr int kLoads = (BM + BN) * KS / 4096;     // loads of a wavefront and stage (1 KiB each)
    static constexpr int kStage = (BM + BN) * KS;            // bytes
    static constexpr int kRows = 1024 / KS;                  // rows of a load
    static constexpr int kChunksRow = KS / 16;               // 16-byte chunks of a row and stage
    static constexpr int kBankRows = 256 / KS;               // rows of the 64 banks
    static constexpr int kScales = S * kStage;               // the tile's scales, behind the stages
    static constexpr int kLds = kScales + (BM + BN) * 4;
    // A step has NS sub-steps of 32 bytes of k.  During sub-step FA all operands of the step that are
    // still in LDS are read; behind it the stage is free, and its refill is issued over SP matrix
    // instructions.
    static constexpr int kNS = KS / 32, kMfma = kTM * kTN;
    static constexpr int slot(int i) { return i * SP / kLoads; }
    static constexpr int issued(int slots) {   // loads of a refill issued before the slot
        int n = 0;
        for (int i = 0; i < kLoads; ++i) n += slot(i) < slots;
        return n;
    }
};

// The workgroup's tile.  Workgroups go round the 8 XCDs; each XCD gets a contiguous run of tiles, taken
// kGroup tile rows at a time, so that the tiles an XCD works on at once share rows in its L2.
constexpr int kXcds = 8, kGroup = 8;
__device__ __forceinline__ int tile_of(int b, int splits, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int tiles = tiles_m * tiles_n, all = tiles * splits, per = all / kXcds, rest = all % kXcds, x = b % kXcds;
    int t = x * per + (x < rest ? x : rest) + b / kXcds;
    const int split = t / tiles;
    t -= split * tiles;
    const int group = t / (kGroup * tiles_n), first = group * kGroup;
    const int in = tiles_m - first < kGroup ? tiles_m - first : kGroup, at = t - first * tiles_n;
    tm = first + at % in;
    tn = at / in;
    return split;
}

template <int BM, int BN, int WM, int KS, int S, int SP, int FA, int OUT>
__global__ __launch_bounds__(256, 1) void k_gemm8(Gemm8Args a, int tiles_m, int tiles_n, int splits) {
    using C = TileCfg<BM, BN, WM, KS, S, SP, FA>;
    constexpr int TM = C::kTM, TN = C::kTN;
    // a refill ends before the next one begins; vmcnt counts to 63; a thread clears at most one row's tail
    static_assert(SP <= C::kNS * C::kMfma && S * C::kLoads < 64 && BM <= 256 && S >= 2 && C::kNS % 2 == 0);
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    int tile_m, tile_n;
    const int split = tile_of(blockIdx.x, splits, tiles_m, tiles_n, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * BM, n0 = (int64_t)tile_n * BN;
    const int rows_m = a.M - tile_m * BM < BM ? a.M - tile_m * BM : BM;
    const int rows_n = a.N - tile_n * BN < BN ? a.N - tile_n * BN : BN;
    // this workgroup's part of k: steps first .. first + steps - 1
    const int all_steps = (a.K + KS - 1) / KS, pad_k = (a.K + 15) / 16 * 16;
    const int first = (int)((int64_t)all_steps * split / splits);
    const int steps = (int)((int64_t)all_steps * (split + 1) / splits) - first;

    // Loads.  One moves 8 rows of 128 bytes; LDS row r holds its 16-byte chunk c at place c ^ (r / 2 % 8).
    // A 16-byte read goes through LDS in phases of 16 lanes over 64 banks, here 16 rows at one c: 8 even
    // ones in one half of the banks and 8 odd ones in the other, each at a place of its own (with
    // c ^ (r % 8) pairs of rows of a phase met, and reads took 1.5 times as long).
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    constexpr int kLoadsX = BM * KS / 4096;
    uint32_t voff[C::kLoads];
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
        const bool is_x = i < kLoadsX;
        const int row = ((is_x ? i : i - kLoadsX) * 4 + wave) * C::kRows + lane / C::kChunksRow;
        voff[i] = (uint32_t)row * (uint32_t)(is_x ? a.ld_x : a.ld_w) +
                  (uint32_t)((lane % C::kChunksRow) ^ (row / C::kBankRows % C::kChunksRow)) * 16;
    }
    const uint64_t base_x = (uint64_t)(a.xq + m0 * a.ld_x + (int64_t)first * KS);
    const uint64_t base_w = (uint64_t)(a.wq + n0 * a.ld_w + (int64_t)first * KS);
    const uint32_t size_x = (uint32_t)((rows_m - 1) * a.ld_x) + pad_k - first * KS;
    const uint32_t size_w = (uint32_t)((rows_n - 1) * a.ld_w) + pad_k - first * KS;
    // The buffers of step t: they end with the tile's last row, and are empty past the last step.  Loads past
    // them touch no memory; the count of loads under way is the same in every step.
    auto rsrc = [&](uint64_t base, uint32_t size, int t) {
        return rsrc_of(base + (uint64_t)t * KS, t < steps ? size - (uint32_t)t * KS : 0u);
    };
    auto load = [&](int i, u32x4 rx, u32x4 rw, uint32_t stage) {
        const bool is_x = i < kLoadsX;
        load_lds16(is_x ? rx : rw, voff[i], stage + (uint32_t)(i * 4 + wave) * 1024);
    };
    // Bytes past K of the last step's activations become zeros.
    auto clear_tail = [&](uint8_t* st) {
        const int row = threadIdx.x, at = a.K % KS;
#pragma unroll 1
        for (int c = row < BM ? at / 16 : C::kChunksRow; c < C::kChunksRow; ++c) {
            uint8_t* p = st + row * KS + (c ^ (row / C::kBankRows % C::kChunksRow)) * 16;
            if (c * 16 >= at) {
                *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
            } else {
                for (int k = at % 16; k < 16; ++k) p[k] = 0;
            }
        }
        wait_reads();
    };
    const bool tail = a.K % KS != 0 && split + 1 == splits;

    // Operands: block row lane % 32, 16-byte chunk 2 ks + lane / 32 of sub-step ks.
    const int wm = wave / C::kWN, wn = wave % C::kWN;
    constexpr int NS = C::kNS;
    uint32_t col[NS];
#pragma unroll
    for (int ks = 0; ks < NS; ++ks)
        col[ks] = (lane % 32) * KS + (((2 * ks + lane / 32) ^ (lane / C::kBankRows % C::kChunksRow)) * 16);
    const uint32_t row_x = wm * C::kRowsM * KS, row_w = (BM + wn * C::kRowsN) * KS;
    i32x4 fx[NS][TM], fw[NS][TN];
    auto read = [&](int i, int set, const uint8_t* st, int ks) {
        if (i < TN)
            fw[set][i] = *reinterpret_cast<const i32x4*>(st + row_w + i * 32 * KS + col[ks]);
        else
            fx[set][i - TN] = *reinterpret_cast<const i32x4*>(st + row_x + (i - TN) * 32 * KS + col[ks]);
    };
    i32x16 acc[TN][TM];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[n][m] = (i32x16)(0);

    // the scales of the tile wait in registers until the stages are no longer needed
    constexpr int kScaleRegs = (BM + BN + 255) / 256;
    float scale[kScaleRegs];
#pragma unroll
    for (int i = 0; i < kScaleRegs; ++i) {
        const int at = i * 256 + (int)threadIdx.x, n = at - BM;
        scale[i] = 0.0f;
        if (at < BM) scale[i] = a.xs[m0 + (at < rows_m ? at : rows_m - 1)];
        else if (n < BN) scale[i] = a.ws[n0 + (n < rows_n ? n : rows_n - 1)];
    }

    // The first S - 1 stages, and of the next one what a step issues before it ends.
    constexpr int kRefillStart = (NS - 1 - FA) * C::kMfma;   // slots of a refill within its own step
    u32x4 rx, rw;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        rx = rsrc(base_x, size_x, s);
        rw = rsrc(base_w, size_w, s);
        asm volatile("s_nop 4" ::"s"(rx), "s"(rw));
#pragma unroll
        for (int i = 0; i < (s < S - 1 ? C::kLoads : C::issued(kRefillStart)); ++i)
            load(i, rx, rw, lds0 + s * C::kStage);
    }
    wait_stage<(S - 2) * C::kLoads + C::issued(kRefillStart)>();
    if (steps == 1 && tail) clear_tail(lds);
#pragma unroll
    for (int i = 0; i < TM + TN; ++i) read(i, 0, lds, 0);

    int buf = 0, refill = S - 1;
    for (int t = 0; t < steps; ++t) {
        const int next = buf + 1 < S ? buf + 1 : 0;
        const uint8_t* cur_p = lds + buf * C::kStage;
        uint8_t* next_p = lds + next * C::kStage;
        static_for<NS>([&](auto ks_) {
            constexpr int ks = ks_;
            if constexpr (ks == FA + 1) {
                // every wavefront has read this stage: its refill may begin
                if constexpr (ks < NS - 1) wait_reads();
                else wait_stage<(S - 2) * C::kLoads + C::issued(kRefillStart - C::kMfma)>();
                rx = rsrc(base_x, size_x, t + S);
                rw = rsrc(base_w, size_w, t + S);
                refill = buf;
                // a scalar register written by a vector instruction needs five wait states before a load
                // reads it; the compiler does not look into the assembly of the loads
                asm volatile("s_nop 4" ::"s"(rx), "s"(rw));
            } else if constexpr (ks == NS - 1) {
                wait_stage<(S - 2) * C::kLoads + C::issued(kRefillStart - C::kMfma)>();
            }
            if (ks == NS - 1 && tail && t + 2 == steps) clear_tail(next_p);
            constexpr int kOps = TM + TN;
            constexpr int reads = ks < FA || ks == NS - 1 ? kOps : ks == FA ? (NS - 1 - FA) * kOps : 0;
            static_for<C::kMfma>([&](auto j_) {
                constexpr int j = j_;
                static_for<reads>([&](auto i) {
                    constexpr int at = reads > C::kMfma ? i * C::kMfma / reads : int(i), set = (ks + 1 + i / kOps) % NS;
                    if constexpr (at == j) read(i % kOps, set, ks == NS - 1 ? next_p : cur_p, set);
                });
                constexpr int slot = ((ks + NS - 1 - FA) % NS) * C::kMfma + j;
                static_for<C::kLoads>([&](auto i) {
                    if constexpr (C::slot(i) == slot) load(i, rx, rw, lds0 + refill * C::kStage);
                });
                constexpr int n = j / TM, m = j % TM;
                acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[ks][n], fx[ks][m], acc[n][m], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        buf = next;
    }

    // Rows of y through LDS, 32 at a time and wavefront, for stores of whole lines.  A lane has column
    // m = lane % 32 of each block and rows n = 8 g + 4 (lane / 32) + 0..3.
    float* scales = reinterpret_cast<float*>(lds + C::kScales);
#pragma unroll
    for (int i = 0; i < kScaleRegs; ++i)
        if (i * 256 + (int)threadIdx.x < BM + BN) scales[i * 256 + threadIdx.x] = scale[i];
    wait_stage<0>();
    constexpr int kEs = OUT == kBf16 ? 2 : 4, kRow = C::kRowsN * kEs, kChunks = kRow / 16;
    constexpr int kParts = C::kScales / (4 * 32 * kRow) < TM ? C::kScales / (4 * 32 * kRow) : TM;
    const int r = lane % 32, h = lane / 32;
    float4 ws[TN][4];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            ws[n][g] = *reinterpret_cast<const float4*>(scales + BM + wn * C::kRowsN + n * 32 + 8 * g + 4 * h);
    const int64_t pitch = (OUT == kSums ? (int64_t)sums_pitch(a.N) : a.ld_y) * kEs;
    const bool full = rows_m == BM && rows_n == BN;
    uint8_t* out = reinterpret_cast<uint8_t*>(OUT == kSums ? a.work : a.y);
    if (OUT == kSums) out += (int64_t)split * a.M * pitch;
    uint8_t* y = out + (m0 + wm * C::kRowsM) * pitch + (n0 + wn * C::kRowsN) * kEs;
    uint8_t* y_lane = y + (lane / kChunks) * pitch + (lane % kChunks) * 16;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        uint8_t* mine = lds + (m % kParts * 4 + wave) * 32 * kRow;
        const float xs = scales[wm * C::kRowsM + m * 32 + r];
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int byte = (n * 32 + 8 * g + 4 * h) * kEs;
                uint8_t* p = mine + r * kRow + (((byte / 16) ^ r) % kChunks) * 16 + byte % 16;
                if constexpr (OUT == kSums) {
                    *reinterpret_cast<i32x4*>(p) = i32x4{acc[n][m][4 * g], acc[n][m][4 * g + 1],
                                                         acc[n][m][4 * g + 2], acc[n][m][4 * g + 3]};
                    continue;
                }
                const float4 w = ws[n][g];
                const float v[4] = {(float)acc[n][m][4 * g] * xs * w.x, (float)acc[n][m][4 * g + 1] * xs * w.y,
                                    (float)acc[n][m][4 * g + 2] * xs * w.z, (float)acc[n][m][4 * g + 3] * xs * w.w};
                if constexpr (OUT == kBf16)
                    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
                else
                    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            }
        constexpr int kStores = 32 * kChunks / kWave, kRowsStore = kWave / kChunks;
        const int c = lane % kChunks;
        if (full) {
#pragma unroll
            for (int i = 0; i < kStores; ++i) {
                const int row = i * kRowsStore + lane / kChunks;
                *reinterpret_cast<Out16*>(y_lane + (m * 32 + i * kRowsStore) * pitch) =
                    *reinterpret_cast<const Out16*>(mine + row * kRow + ((c ^ row) % kChunks) * 16);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kStores; ++i) {
                const int row = i * kRowsStore + lane / kChunks;
                const int left = rows_n - wn * C::kRowsN - c * (16 / kEs);
                const uint8_t* p = mine + row * kRow + ((c ^ row) % kChunks) * 16;
                uint8_t* to = y_lane + (m * 32 + i * kRowsStore) * pitch;
                if (wm * C::kRowsM + m * 32 + row >= rows_m || left <= 0) continue;
                if (left >= 16 / kEs) {
                    *reinterpret_cast<Out16*>(to) = *reinterpret_cast<const Out16*>(p);
                } else {
                    for (int e = 0; e < left; ++e) {
                        if constexpr (OUT == kBf16)
                            reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(p)[e];
                        else
                            reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(p)[e];
                    }
                }
            }
        }
    }
}

// Adds the sums of the parts of k: 4 columns of a row a thread.
template <bool BF>
__global__ __launch_bounds__(256) void k_gemm8_join(Gemm8Args a, int splits) {
    const int pitch = sums_pitch(a.N), quads = (a.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / quads;
    const int n = (int)(i % quads) * 4;
    if (m >= a.M) return;
    const int* p = reinterpret_cast<const int*>(a.work) + m * pitch + n;
    i32x4 c = *reinterpret_cast<const i32x4*>(p);
    int s = 1;
    for (; s + 3 <= splits; s += 3) {   // three loads under way at a time
        i32x4 v[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) v[u] = *reinterpret_cast<const i32x4*>(p + (int64_t)(s + u) * a.M * pitch);
#pragma unroll
        for (int u = 0; u < 3; ++u) c += v[u];
    }
    for (; s < splits; ++s) c += *reinterpret_cast<const i32x4*>(p + (int64_t)s * a.M * pitch);
    const float xs = a.xs[m];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)c[e] * xs * a.ws[n + e < a.N ? n + e : n];
    if constexpr (BF) {
        uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * a.ld_y + n;
        const Out8 o = {{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}};
        if (n + 4 <= a.N)
            *reinterpret_cast<Out8*>(y) = o;
        else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < a.N) y[e] = (uint16_t)(o.w[e / 2] >> (16 * (e % 2)));
        }
    } else {
        float* y = reinterpret_cast<float*>(a.y) + m * a.ld_y + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) y[e] = v[e];
    }
}

// Lets a kernel use more than the default 64 KiB of LDS on the current device; `done` has a bit for each
// device where that has been said.
template <typename K>
hipError_t allow_big_lds(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    else (void)hipGetLastError();
    return e;
}

template <int BM, int BN, int WM, int KS, int S, int SP, int FA, int OUT>
hipError_t launch_tile_kernel(const Gemm8Args& a, int tiles_m, int tiles_n, int splits, hipStream_t st) {
    using C = TileCfg<BM, BN, WM, KS, S, SP, FA>;
    auto kernel = k_gemm8<BM, BN, WM, KS, S, SP, FA, OUT>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_big_lds(kernel, C::kLds, done);
    if (e != hipSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)(tiles_m * tiles_n * splits)), 256, C::kLds, st, a, tiles_m, tiles_n,
                         splits);
}

template <int BM, int BN, int WM, int KS, int S, int SP, int FA>
hipError_t launch_tiles(const Gemm8Args& a, hipStream_t st) {
    const int tiles_m = (int)(((int64_t)a.M + BM - 1) / BM), tiles_n = (int)(((int64_t)a.N + BN - 1) / BN);
    return a.y_bf16 ? launch_tile_kernel<BM, BN, WM, KS, S, SP, FA, kBf16>(a, tiles_m, tiles_n, 1, st)
                    : launch_tile_kernel<BM, BN, WM, KS, S, SP, FA, kF32>(a, tiles_m, tiles_n, 1, st);
}

// The same, or with k in parts and their join.
template <int BM, int BN, int WM, int KS, int S, int SP, int FA>
hipError_t launch_tiles_or_parts(const Gemm8Args& a, int splits, hipStream_t st) {
    if (splits == 1) return launch_tiles<BM, BN, WM, KS, S, SP, FA>(a, st);
    const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    const hipError_t e = launch_tile_kernel<BM, BN, WM, KS, S, SP, FA, kSums>(a, tiles_m, tiles_n, splits, st);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(((int64_t)a.M * ((a.N + 3) / 4) + 255) / 256));
    return launch_kernel(a.y_bf16 ? k_gemm8_join<true> : k_gemm8_join<false>, grid, 256, 0, st, a, splits);
}

// Few activation rows: bound by the one read of the weights.  A workgroup has up to 32 weight rows, as many
// as spread the matrix evenly over the compute units, and W wavefronts that split k between them.  Each
// wavefront runs on its own: it loads 128 bytes of k of all rows (a unit) at a time into its own ring of S
// units in LDS (XL loads of 8 activation rows, 4 of weight rows), and waits for nothing but its own loads.
template <int W, int S, int XL, int OUT>
__global__ __launch_bounds__(W * kWave) void k_gemm8_thin(Gemm8Args a, int rows) {
    constexpr int MT = XL > 4 ? 2 : 1, kUnit = (4 + XL) * 1024, kLoads = 4 + XL;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = blockIdx.x * rows, rows_n = a.N - n0 < rows ? a.N - n0 : rows, pad_k = (a.K + 15) / 16 * 16;
    const int units = (a.K + 127) / 128, u0 = units * wave / W, u1 = units * (wave + 1) / W;
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds + wave * S * kUnit;
    const uint8_t* ring_p = lds + wave * S * kUnit;
    uint32_t voff[kLoads];   // the layout of a stage of a tile, weight rows first
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = (i < 4 ? i : i - 4) * 8 + lane / 8;
        voff[i] = (uint32_t)row * (uint32_t)(i < 4 ? a.ld_w : a.ld_x) + (uint32_t)((lane % 8) ^ (row / 2 % 8)) * 16;
    }
    const uint64_t base_w = (uint64_t)(a.wq + (int64_t)n0 * a.ld_w), base_x = (uint64_t)a.xq;
    const uint32_t size_w = (uint32_t)(rows_n - 1) * (uint32_t)a.ld_w + pad_k;
    const uint32_t size_x = (uint32_t)(a.M - 1) * (uint32_t)a.ld_x + pad_k;
    auto load = [&](int u, int slot) {   // past the wavefront's part: from empty buffers
        const uint32_t at = (uint32_t)u * 128;
        const u32x4 rw = rsrc_of(base_w + at, u < u1 ? size_w - at : 0);
        const u32x4 rx = rsrc_of(base_x + at, u < u1 ? size_x - at : 0);
        asm volatile("s_nop 4" ::"s"(rw), "s"(rx));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_lds16(i < 4 ? rw : rx, voff[i], ring + slot * kUnit + i * 1024);
    };
#pragma unroll
    for (int s = 0; s < S; ++s) load(u0 + s, s);
    uint32_t col[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) col[ks] = (lane % 32) * 128 + (((2 * ks + lane / 32) ^ (lane / 2 % 8)) * 16);
    i32x16 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = (i32x16)(0);
    int slot = 0;
    for (int u = u0; u < u1; ++u) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * kLoads) : "memory");
        const uint8_t* p = ring_p + slot * kUnit;
        i32x4 fw[4], fx[4][MT];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            fw[ks] = *reinterpret_cast<const i32x4*>(p + col[ks]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // with fewer than 32 rows of activations in the ring, columns past them repeat its first rows
                const int wrap = XL < 4 ? XL * 1024 - 1 : 8191;
                fx[ks][m] = *reinterpret_cast<const i32x4*>(p + 4096 + ((m * 4096 + col[ks]) & wrap));
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: refill it
        load(u + S, slot);
        const int left = a.K - u * 128 - lane / 32 * 16;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if ((u + 1) * 128 > a.K) {   // bytes past K are not part of a row
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int n = left - ks * 32 - d * 4;
                        if (n < 4) fx[ks][m][d] = n <= 0 ? 0 : fx[ks][m][d] & ((1 << (8 * n)) - 1);
                    }
                }
                acc[m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[ks], fx[ks][m], acc[m], 0, 0, 0);
            }
        slot = slot + 1 < S ? slot + 1 : 0;
    }
    wait_stage<0>();
    int* part = reinterpret_cast<int*>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) part[((wave * MT + m) * 16 + i) * kWave + lane] = acc[m][i];
    __syncthreads();
    for (int o = threadIdx.x; o < a.M * 32; o += W * kWave) {
        const int m = o / 32, n = o % 32;
        if (n >= rows_n) continue;
        const int* p = part + (m / 32 * 16 + n / 8 * 4 + n % 4) * kWave + n / 4 % 2 * 32 + m % 32;
        int c = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) c += p[w * MT * 16 * kWave];
        const float y = (float)c * a.xs[m] * a.ws[n0 + n];
        const int64_t at = m * a.ld_y + n0 + n;
        if constexpr (OUT == kBf16)
            reinterpret_cast<uint16_t*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)y);
        else
            reinterpret_cast<float*>(a.y)[at] = y;
    }
}

template <int W, int S, int XL, int OUT>
hipError_t launch_thin_kernel(const Gemm8Args& a, hipStream_t st) {
    constexpr int MT = XL > 4 ? 2 : 1, kRing = W * S * (4 + XL) * 1024, kPart = W * MT * 4096;
    constexpr int kLds = kRing > kPart ? kRing : kPart;
    const int rows = thin_rows(a.N);
    auto kernel = k_gemm8_thin<W, S, XL, OUT>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_big_lds(kernel, kLds, done);
    if (e != hipSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)((a.N + rows - 1) / rows)), W * kWave, kLds, st, a, rows);
}

// 4 wavefronts, and as many units in flight as leave room for two workgroups a compute unit (up to 32
// activation rows).
template <int OUT>
hipError_t launch_thin(const Gemm8Args& a, hipStream_t st) {
    if (a.M <= 8) return launch_thin_kernel<4, 3, 1, OUT>(a, st);
    if (a.M <= 16) return launch_thin_kernel<4, 3, 2, OUT>(a, st);
    if (a.M <= 32) return launch_thin_kernel<4, 2, 4, OUT>(a, st);
    return launch_thin_kernel<4, 2, 8, OUT>(a, st);
}

}  // namespace

size_t gemm8_workspace(int M, int N, int K) {
    if (M == 0 || N == 0) return 0;
    const Plan p = plan(M, N, K);
    return p.splits > 1 ? (size_t)p.splits * M * sums_pitch(N) * 4 : 0;
}

hipError_t launch_gemm8(const Gemm8Args& a, hipStream_t st) {
    const Plan p = plan(a.M, a.N, a.K);
    switch (p.tile) {
    case 0: return launch_tiles<256, 256, 2, 128, 2, 48, 0>(a, st);
    case 1: return launch_tiles_or_parts<256, 128, 2, 128, 3, 32, 0>(a, p.splits, st);
    case 2: return launch_tiles_or_parts<128, 128, 2, 128, 4, 16, 0>(a, p.splits, st);
    case 3: return launch_tiles_or_parts<128, 64, 4, 128, 6, 8, 0>(a, p.splits, st);
    case 4: return launch_tiles_or_parts<64, 128, 2, 128, 6, 8, 0>(a, p.splits, st);
    case 5: return launch_tiles_or_parts<64, 64, 2, 128, 8, 4, 0>(a, p.splits, st);
    default: return a.y_bf16 ? launch_thin<kBf16>(a, st) : launch_thin<kF32>(a, st);
    }
}

}  // namespace qamw
