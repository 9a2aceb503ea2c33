// Products of matrices of 4-bit codes with a power of two for every 32 columns: y[m][n] = sum_k x[m][k] w[n][k], on
// the matrix cores (v_mfma_scale_f32_32x32x64_f8f6f4), and the same for rows in groups with weights of their own.
//
// An operand of the instruction is one block of 32 columns a lane, with the block's scale byte: lane l has row l % 32,
// and lanes 0-31 and 32-63 have two different blocks.  Which blocks does not matter as long as both operands agree:
// of a group of 8 blocks the lower lanes have 0-3 and the upper ones 4-7, so that a lane's four scale bytes are
// the four bytes of a register, from which the instruction takes the one that it is told.
//
// Two kernels.  k_gemm4 forms tiles of y, with the operands in stages of a group of 256 columns in LDS; where the tiles
// do not fill the chip, k is split over workgroups too and k_gemm4_join adds their sums, in fp32 and in the order of
// k.  k_gemm4_thin, for few activation rows, is bound by one read of the weights.  Both have a form for rows in groups.
// plan4() and plan4_grouped() (qamw_mx4_plan.hpp) choose.
//
// Loads.  A stage is 128 bytes of codes of every row, whole lines of memory, and 8 bytes of scales, which stand together
// for the rows of a tile (groups are the outermost dimension of the scales): with scales by rows a stage would fetch
// 64 bytes of them for every 8.  Everything goes from memory straight to LDS; rows and columns past the end come
// from the buffer's bounds as zeros, code and scale alike, so there are no masks.
#include "qamw_device.hpp"
#include "qamw_mx4_launch.hpp"
#include "qamw_mx4_plan.hpp"
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

// Rows in groups.  Tiles of `bm` rows are counted over all groups, each group beginning a tile of its own.  What the
// groups are is known to the device only: a launch has workgroups for as many tiles as there may be, and those
// without one leave.  Every wavefront counts by itself, 64 groups at a time, a group a lane.
struct Groups {
    int lo, hi, sum;   // the lane's group, held to the rows there are, and the tiles up to its end
};
__device__ __forceinline__ Groups groups_from(const Gemm4Args& a, int bm, int e) {
    Groups g{0, 0, 0};
    if (e < a.experts) {
        const int lo = a.offsets[e], hi = a.offsets[e + 1];
        g.lo = lo < 0 ? 0 : lo > a.M ? a.M : lo;
        g.hi = hi < 0 ? 0 : hi > a.M ? a.M : hi;
    }
    g.sum = g.hi > g.lo ? (g.hi - g.lo + bm - 1) / bm : 0;
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const int below = __shfl_up(g.sum, off);
        g.sum += (int)threadIdx.x % kWave >= off ? below : 0;
    }
    return g;
}
// Which tile a workgroup has: rows m0 .. m0 + rows_m - 1, columns n0 .. n0 + rows_n - 1, part `split` of k, an expert.
struct Tile {
    int m0, rows_m, n0, rows_n, split, expert;
};
// The tiles of a launch in their order.
template <int BM, int BN, bool GROUPED>
struct Tiles {
    Groups g;             // the last 64 groups counted (of up to 64, all)
    int tiles_m, tiles_n, splits, count;
    __device__ __forceinline__ Tiles(const Gemm4Args& a, int tm, int tn, int sp) : g{}, tiles_m(tm), tiles_n(tn), splits(sp) {
        if constexpr (GROUPED) {
            int total = 0;
            for (int e0 = 0; e0 < a.experts; e0 += kWave) {
                g = groups_from(a, BM, e0 + (int)threadIdx.x % kWave);
                total += __shfl(g.sum, kWave - 1);
            }
            total = __builtin_amdgcn_readfirstlane(total);
            tiles_m = total < tiles_m ? total : tiles_m;   // (more only where groups overlap)
        }
        count = tiles_m * tiles_n * splits;
    }
    __device__ __forceinline__ Tile at(const Gemm4Args& a, int number) {
        Tile t{};
        int tile_m, tile_n;
        t.split = tile_of(number, splits, tiles_m, tiles_n, tile_m, tile_n);
        int m_end = a.M;
        if constexpr (GROUPED) {
            m_end = 0;   // (a tile without rows, should the offsets change under the call)
            for (int e0 = 0; e0 < a.experts; e0 += kWave) {
                if (a.experts > kWave) g = groups_from(a, BM, e0 + (int)threadIdx.x % kWave);
                const uint64_t reached = __ballot(g.sum > tile_m);
                if (reached) {
                    const int lane = __builtin_ctzll(reached);
                    const int before = lane > 0 ? __shfl(g.sum, lane - 1) : 0;
                    t.expert = __builtin_amdgcn_readfirstlane(e0 + lane);
                    m_end = __builtin_amdgcn_readfirstlane(__shfl(g.hi, lane));
                    t.m0 = __builtin_amdgcn_readfirstlane(__shfl(g.lo, lane) + (tile_m - before) * BM);
                    break;
                }
                tile_m -= __shfl(g.sum, kWave - 1);
            }
        } else {
            t.m0 = tile_m * BM;
        }
        t.n0 = tile_n * BN;
        t.rows_m = m_end - t.m0 < BM ? m_end - t.m0 : BM;
        t.rows_n = a.N - t.n0 < BN ? a.N - t.n0 : BN;
        return t;
    }
};

// 4 bytes a lane from a buffer into LDS at lds + 4 lane, like load_lds16.
__device__ __forceinline__ void load_lds4(u32x4 rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory");
}

// What a tile leaves: y, or its sums over a part of k, to be joined.
enum { kF32 = 0, kBf16 = 1, kSums = 2 };

// A tile of BM activation rows by BN weight rows, WM x 4 / WM wavefronts, S stages of a group of columns in LDS: the
// rows' 128 bytes of codes, then their 8 bytes of scales.
//
// What bounds it.  256 x 256 of a group are 64 matrix instructions of 32 cycles for each of the 4 SIMDs, 2099 cycles, in
// which LDS delivers 128 KiB to the operands and takes in 68.  At 8192 x 13824 x 5120 a step takes 2670 cycles (2590 with
// empty buffers; 2970 while the output went through the cache), at 1.71 GHz: the chip's power is the limit, and what
// moves data takes its part of it.  Matrix instructions from registers alone reach 6.75 PFLOP/s on codes of normal
// values (9.2 on zeros, at 2.3 GHz); here 4.4.  Smaller tiles have fewer matrix cycles for the bytes that LDS
// moves: a step of 128 x 128 is 525 matrix cycles and 770 of LDS, and takes 870 with empty buffers.
//   step by step (us, that size): operands as they stand in memory, no LDS 2557; tiles through LDS, one tile a workgroup
//   289 (of 70000 cycles a tile 8000 until the first stage is there and 7400 for the output); conversions to bf16 in
//   pairs 281; workgroups that walk over tiles 276 to 290 on cards where the form before takes 281 to 293 (the cycles
//   fall by 10%, the clock by 6%); streaming stores of the output, so that the operands that other tiles read stay in the
//   cache, 261 where the form before takes 273 to 276 (128 x 256 tiles 388 -> 309; 16384 x 4096 x 2048 83 -> 80).  That
//   is with three sets of operands by turns; with one set, and with what reads the output behind it (quant4, gated), us,
//   stored ordinarily and streaming: 1024 x 8192 x 4096 30.5 and 30.2, 2048 x 22016 x 4096 130 and 134, 4096 x 27648 x
//   5120 381 and 358; 8192 rows in 16 groups, 8192 x 2048, 161 and 170: neither is better for all sizes.
//   Back to back the chip's power holds for 6 of these products only (263), then they take up to 370 and settle at 305.
//   Not kept: the stage's operands read over two or three sub-steps instead of one (+1%, +12%); a refill
//   over 32 (+2%) or 60 (-1%, but then a walk's stores stand before loads) instructions; all sums of a part read
//   before the first conversion (+11%: scratch memory).
template <int BM, int BN, int WM, int S, int SP>
struct TileCfg {
    static constexpr int kWN = 4 / WM, kRowsM = BM / WM, kRowsN = BN / kWN;   // a wavefront's part
    static constexpr int kTM = kRowsM / 32, kTN = kRowsN / 32;                // in blocks of 32 x 32
    static constexpr int kCodeLoads = (BM + BN) / 32;        // loads of a wavefront and stage: 8 rows of codes each
    static constexpr int kScaleRows = (BM + BN) / 32;        // 32 rows of scales each, for the workgroup
    static constexpr int kScaleLoads = (kScaleRows + 3) / 4;
    static constexpr int kLoads = kScaleLoads + kCodeLoads;
    static constexpr int kCodes = (BM + BN) * kGroupBytes, kStage = kCodes + (BM + BN) * 8, kLds = S * kStage;
    // A step has 4 sub-steps of two blocks a row.  Its refill is issued over SP matrix instructions.
    static constexpr int kNS = 4, kMfma = kTM * kTN;
    static constexpr int slot(int i) { return i * SP / kLoads; }
    static constexpr int issued(int slots) {   // loads of a refill issued before the slot
        int n = 0;
        for (int i = 0; i < kLoads; ++i) n += slot(i) < slots;
        return n;
    }
};

constexpr uint32_t kFar = 0xF0000000u;   // an offset past every buffer: what is loaded from there is 0

// Waits until at most N of the wavefront's loads and stores are under way; where the output of the tile before was
// stored with STORES stores behind the loads that are waited for, those may be under way too.
template <int N, int STORES>
__device__ __forceinline__ void wait_stage_behind(bool stored) {
    if constexpr (STORES > 0 && N + STORES < 64) {
        if (stored) {
            wait_stage<N + STORES>();
            return;
        }
    }
    wait_stage<N>();
}

// A kernel's first argument, read from memory again: what a loop needs only now and then is not kept in scalar
// registers, which would not suffice (and a spilled one costs a vector instruction each time).  They do not suffice all
// the same: the walk has 12 (fp32 output) and 22 (bf16) spilled ones, in groups 50 and 59, most of them used where a
// tile begins or ends.
__device__ __forceinline__ Gemm4Args args_again() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Gemm4Args*)p;
}

// WALK: a workgroup has every gridDim-th tile, one behind the other, and the loads of the next tile's first stages are
// under way while the last ones are multiplied and the output is formed.  Otherwise it has one.
template <int BM, int BN, int WM, int S, int SP, int OUT, bool GROUPED, bool WALK>
__global__ __launch_bounds__(256, 1) void k_gemm4(Gemm4Args a, int tiles_m, int tiles_n, int splits) {
    using C = TileCfg<BM, BN, WM, S, SP>;
    constexpr int TM = C::kTM, TN = C::kTN, NS = C::kNS;
    // a refill ends before the next one begins; vmcnt counts to 63
    static_assert(SP <= NS * C::kMfma && S * C::kLoads < 64 && S >= 2);
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Tiles<BM, BN, GROUPED> tiles(a, tiles_m, tiles_n, splits);
    int number = blockIdx.x;
    if (number >= tiles.count) return;
    Tile tile = tiles.at(a, number);

    // Loads.  One moves 8 rows of 128 bytes; LDS row r holds its 16-byte chunk c at place c ^ (r / 2 % 8).
    // A 16-byte read goes through LDS in phases of 16 lanes over 64 banks, here 16 rows at one c: 8 even
    // ones in one half of the banks and 8 odd ones in the other, each at a place of its own.
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    constexpr int kLoadsX = BM / 32;
    const bool indexed = GROUPED && a.index;
    uint32_t voff[C::kLoads];   // scales first
    // The offsets in x go by the tile where rows have an index, and by the place in the tile alone otherwise.  A
    // wavefront loads codes of (up to) 64 rows and scales of 64: a lane fetches the index of one of either, and the
    // others ask it.
    auto offsets = [&](const Gemm4Args& a, const Tile& at, bool of_x_only) {
        uint32_t lane = threadIdx.x % kWave;
        int of_codes = 0, of_scales = 0;
        asm volatile("" : "+v"(lane));   // what follows from it is formed here, and takes no registers in the loop
        auto fetch = [&](uint32_t r) { return a.index[at.m0 + ((int)r < at.rows_m ? (int)r : 0)]; };
        if (indexed) {
            of_codes = fetch((lane / 8 * 4 + wave) * 8 + lane % 8);
            of_scales = fetch((lane / 32 * 4 + wave) * 32 + lane % 32);
        }
        auto far = [&](uint32_t r, int row) { return (int)r >= at.rows_m || row < 0 || row >= a.x_rows; };
#pragma unroll
        for (int i = 0; i < C::kScaleLoads; ++i) {
            const int n = i * 4 + wave, part = n < C::kScaleRows ? n : C::kScaleRows - 1;
            const bool is_x = kLoadsX % 4 ? part < kLoadsX : i < kLoadsX / 4;
            if (of_x_only && !is_x) continue;
            const uint32_t r = (uint32_t)(is_x ? part : part - kLoadsX) * 32 + lane / 2;
            voff[i] = r * 8 + lane % 2 * 4;
            if (indexed && is_x) {
                const int row = __shfl(of_scales, i * 32 % kWave + lane / 2);
                voff[i] = far(r, row) ? kFar : (uint32_t)row * 8 + lane % 2 * 4;
            }
        }
#pragma unroll
        for (int i = 0; i < C::kCodeLoads; ++i) {
            const bool is_x = i < kLoadsX;
            if (of_x_only && !is_x) continue;
            const uint32_t r = (uint32_t)((is_x ? i : i - kLoadsX) * 4 + wave) * 8 + lane / 8;
            const uint32_t chunk = ((lane % 8) ^ (r / 2 % 8)) * 16;
            uint32_t& v = voff[C::kScaleLoads + i];
            v = r * (uint32_t)(is_x ? a.ld_x : a.ld_w) + chunk;
            if (indexed && is_x) {
                const int row = __shfl(of_codes, i * 8 % kWave + lane / 8);
                v = far(r, row) ? kFar : (uint32_t)row * (uint32_t)a.ld_x + chunk;
            }
        }
    };
    // Where the next loads come from: step `load_t` of `load_steps` of a tile.  Buffers end with the last row that
    // there is; a row's bytes behind this part of k are in them, and never read.  Behind the last tile they are
    // empty: loads from there touch no memory, and the count of loads under way is the same in every step.
    uint64_t base_x, base_w, base_xe, base_we;
    uint32_t size_x, size_w, size_xe, size_we;
    int load_t, load_steps, load_number = number;
    auto load_from = [&](const Gemm4Args& a, const Tile& at) {
        // (at most 2^15 groups in 8 parts: 32 bits do, and a division of 64 bits takes a thousand cycles)
        const int first = (int)((uint32_t)(a.groups * at.split) / (uint32_t)splits);
        load_steps = (int)((uint32_t)(a.groups * (at.split + 1)) / (uint32_t)splits) - first;
        load_t = 0;
        const int64_t at_m = indexed ? 0 : at.m0, have_x = indexed ? a.x_rows : at.rows_m;
        const uint32_t left = (uint32_t)(a.groups - first) * kGroupBytes;
        base_x = (uint64_t)(a.xq + at_m * a.ld_x + (int64_t)first * kGroupBytes);
        base_w = (uint64_t)(a.wq + (GROUPED ? at.expert * a.ld_wexpert : 0) + at.n0 * a.ld_w + (int64_t)first * kGroupBytes);
        base_xe = (uint64_t)(a.xe + at_m * 8 + first * a.ld_xe);
        base_we = (uint64_t)(a.we + (GROUPED ? at.expert * a.ld_weexpert : 0) + at.n0 * 8ll + first * a.ld_we);
        size_x = have_x ? (uint32_t)((have_x - 1) * a.ld_x) + left : 0;
        size_w = (uint32_t)((at.rows_n - 1) * a.ld_w) + left;
        size_xe = (uint32_t)have_x * 8;
        size_we = (uint32_t)at.rows_n * 8;
    };
    u32x4 rx, rw, rxe, rwe;
    auto buffers = [&]() {   // of the next step
        rx = rsrc_of(base_x, size_x);
        rw = rsrc_of(base_w, size_w);
        rxe = rsrc_of(base_xe, size_xe);
        rwe = rsrc_of(base_we, size_we);
        // a scalar register written by a vector instruction needs five wait states before a load reads it; the
        // compiler does not look into the assembly of the loads
        asm volatile("s_nop 4" ::"s"(rx), "s"(rw), "s"(rxe), "s"(rwe));
        base_x += kGroupBytes;
        base_w += kGroupBytes;
        base_xe += a.ld_xe;
        base_we += a.ld_we;
        size_x = size_x ? size_x - kGroupBytes : 0;
        size_w = size_w ? size_w - kGroupBytes : 0;
    };
    // The buffers of the step behind: of this tile, of the next one, or none.  (Apart from `buffers`, because new
    // offsets may replace the old ones only when the loads that use those have been issued.)
    auto next_step = [&]() {
        if (++load_t < load_steps) return;
        load_number += gridDim.x;
        if (WALK && load_number < tiles.count) {
            const Gemm4Args b = args_again();
            const Tile at = tiles.at(b, load_number);
            load_from(b, at);
            if (indexed) offsets(b, at, true);
        } else {
            size_x = size_w = size_xe = size_we = 0;
            load_t = 0;   // for good: no further tile is looked for
            load_steps = 0x7FFFFFFF;
        }
    };
    auto load = [&](int i, uint32_t stage) {
        if (i < C::kScaleLoads) {
            const int n = i * 4 + wave, part = n < C::kScaleRows ? n : C::kScaleRows - 1;
            // (of the larger tiles, all four wavefronts load of the same operand)
            const bool is_x = kLoadsX % 4 ? part < kLoadsX : i < kLoadsX / 4;
            load_lds4(is_x ? rxe : rwe, voff[i], stage + C::kCodes + (uint32_t)part * 256);
        } else {
            const int j = i - C::kScaleLoads;
            load_lds16(j < kLoadsX ? rx : rw, voff[i], stage + (uint32_t)(j * 4 + wave) * 1024);
        }
    };
    offsets(a, tile, false);
    load_from(a, tile);
    int steps = load_steps;

    // Operands: block row lane % 32, 16-byte chunk ks + 4 (lane / 32) of sub-step ks.
    const int wm = wave / C::kWN, wn = wave % C::kWN;
    uint32_t col[NS];
#pragma unroll
    for (int ks = 0; ks < NS; ++ks)
        col[ks] = (lane % 32) * kGroupBytes + ((ks + lane / 32 * 4) ^ (lane / 2 % 8)) * 16;
    const uint32_t row_x = wm * C::kRowsM * kGroupBytes, row_w = (BM + wn * C::kRowsN) * kGroupBytes;
    const uint32_t scale_x = C::kCodes + (wm * C::kRowsM + lane % 32) * 8 + lane / 32 * 4;
    const uint32_t scale_w = C::kCodes + (BM + wn * C::kRowsN + lane % 32) * 8 + lane / 32 * 4;
    // WALK: during a step's first sub-step, the operands of its others; behind it the stage is free.  Otherwise the
    // operands of a step are read as a whole while the step before is multiplied, so that a step has one barrier and
    // waits for nothing that it has just asked for.
    constexpr int SETS = WALK ? 1 : 2;
    i32x4 fx[SETS * NS][TM], fw[SETS * NS][TN];
    int sx[TM], sw[TN], next_sx[TM], next_sw[TN];
    auto read = [&](int i, int set, const uint8_t* st, int ks) {
        if (i < TN)
            fw[set][i] = *reinterpret_cast<const i32x4*>(st + row_w + i * 32 * kGroupBytes + col[ks]);
        else
            fx[set][i - TN] = *reinterpret_cast<const i32x4*>(st + row_x + (i - TN) * 32 * kGroupBytes + col[ks]);
    };
    auto read_scale = [&](int i, const uint8_t* st) {
        if (i < TN)
            next_sw[i] = *reinterpret_cast<const int*>(st + scale_w + i * 256);
        else
            next_sx[i - TN] = *reinterpret_cast<const int*>(st + scale_x + (i - TN) * 256);
    };

    // The first S - 1 stages, and of the next one what a step issues before it ends.
    constexpr int kRefillStart = WALK ? (NS - 1) * C::kMfma : NS * C::kMfma;   // slots of a refill within its own step
    static_assert(C::issued(kRefillStart) == C::kLoads);   // (the walk's stores are behind whole refills)
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (s > 0) next_step();
        buffers();
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) load(i, lds0 + s * C::kStage);
    }
    constexpr int kOps = TM + TN;
    f32x16 acc[TN][TM];
    if constexpr (!WALK) {   // zeroed while the first loads are under way
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                acc[n][m] = (f32x16)(0.0f);
                asm volatile("" : "+a"(acc[n][m]));
            }
    }
    wait_stage<(S - 1) * C::kLoads>();
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
        read_scale(i, lds);
#pragma unroll
        for (int ks = 0; ks < (WALK ? 1 : NS); ++ks) read(i, ks, lds, ks);
    }

    // Output: 32 rows and 128 bytes of a row (or 64) at a time and wavefront, through LDS for stores of whole lines.
    constexpr int kEs = OUT == kBf16 ? 2 : 4, kPartN = OUT == kBf16 && TN > 1 ? 2 : 1, kRow = kPartN * 32 * kEs;
    constexpr int kChunks = kRow / 16, kStores = 32 * kChunks / kWave, kRowsStore = kWave / kChunks;
    constexpr int kAllStores = TM * TN / kPartN * kStores;   // of a whole tile

    int buf = 0, refill = S - 1;
    bool stored = false;   // the tile before was stored by kAllStores stores
    for (;;) {
        if constexpr (WALK) {
            for (int t = 0; t < steps; ++t) {
                const int next = buf + 1 < S ? buf + 1 : 0;
                const uint8_t* cur_p = lds + buf * C::kStage;
                const uint8_t* next_p = lds + next * C::kStage;
#pragma unroll
                for (int i = 0; i < TN; ++i) sw[i] = next_sw[i];
#pragma unroll
                for (int i = 0; i < TM; ++i) sx[i] = next_sx[i];
                // FIRST: the tile's first products, which are not added to anything
                auto sub_step = [&](auto ks_, auto first_) {
                    constexpr int ks = ks_;
                    constexpr bool FIRST = first_;
                    if constexpr (ks == 1) {
                        // every wavefront has read this stage: its refill may begin
                        wait_reads();
                        next_step();
                        buffers();
                        refill = buf;
                    } else if constexpr (ks == NS - 1) {
                        wait_stage_behind<(S - 2) * C::kLoads + C::issued(kRefillStart - C::kMfma), kAllStores>(stored && t == 0);
                    }
                    constexpr int reads = ks == 0 ? (NS - 1) * kOps : ks == NS - 1 ? kOps : 0;
                    static_for<C::kMfma>([&](auto j_) {
                        constexpr int j = j_;
                        static_for<reads>([&](auto i) {
                            constexpr int at = reads > C::kMfma ? i * C::kMfma / reads : int(i), set = (ks + 1 + i / kOps) % NS;
                            if constexpr (at == j) {
                                read(i % kOps, set, ks == NS - 1 ? next_p : cur_p, set);
                                if constexpr (ks == NS - 1) read_scale(i, next_p);
                            }
                        });
                        constexpr int slot = ((ks + NS - 1) % NS) * C::kMfma + j;
                        static_for<C::kLoads>([&](auto i) {
                            if constexpr (C::slot(i) == slot) load(i, lds0 + refill * C::kStage);
                        });
                        constexpr int n = j / TM, m = j % TM;
                        acc[n][m] = mfma4<ks>(fw[ks][n], fx[ks][m], FIRST ? (f32x16)(0.0f) : acc[n][m], sw[n], sx[m]);
                        __builtin_amdgcn_sched_barrier(0);
                    });
                };
                if (t == 0) sub_step(std::integral_constant<int, 0>{}, std::true_type{});
                else sub_step(std::integral_constant<int, 0>{}, std::false_type{});
                static_for<NS - 1>([&](auto i) { sub_step(std::integral_constant<int, i + 1>{}, std::false_type{}); });
                buf = next;
            }
        } else {
            // The operands of step t are in set SET, or on their way there; step t + 1's go into the other one.
            auto step = [&](auto set_) {
                constexpr int SET = set_;
                const int next = buf + 1 < S ? buf + 1 : 0;
                const uint8_t* next_p = lds + next * C::kStage;
                // every wavefront has read this stage, and the next one is there
                wait_stage<(S - 2) * C::kLoads>();
#pragma unroll
                for (int i = 0; i < TN; ++i) sw[i] = next_sw[i];
#pragma unroll
                for (int i = 0; i < TM; ++i) sx[i] = next_sx[i];
                next_step();
                buffers();
                constexpr int kAll = NS * C::kMfma, kReads = (NS + 1) * kOps;
                static_for<kAll>([&](auto j_) {
                    constexpr int j = j_;
                    static_for<kReads>([&](auto i) {
                        constexpr int at = kReads > kAll ? i * kAll / kReads : int(i);
                        if constexpr (at == j) {
                            if constexpr (i < kOps) read_scale(i, next_p);
                            else read(i % kOps, (1 - SET) * NS + i / kOps - 1, next_p, i / kOps - 1);
                        }
                    });
                    static_for<C::kLoads>([&](auto i) {
                        if constexpr (C::slot(i) == j) load(i, lds0 + buf * C::kStage);
                    });
                    constexpr int ks = j / C::kMfma, n = j % C::kMfma / TM, m = j % TM;
                    acc[n][m] = mfma4<ks>(fw[SET * NS + ks][n], fx[SET * NS + ks][m], acc[n][m], sw[n], sx[m]);
                    __builtin_amdgcn_sched_barrier(0);
                });
                buf = next;
            };
            int t = 0;
            for (; t + 1 < steps; t += 2) {
                step(std::integral_constant<int, 0>{});
                step(std::integral_constant<int, 1>{});
            }
            if (t < steps) step(std::integral_constant<int, 0>{});
        }

        // A lane has column m = lane % 32 of each block and rows n = 8 g + 4 (lane / 32) + 0..3.
        if constexpr (!WALK) wait_stage<0>();   // every stage is free
        uint32_t lane = threadIdx.x % kWave;
        asm volatile("" : "+v"(lane));   // what follows from it is formed here, and takes no registers in the loop
        const uint32_t r = lane % 32, h = lane / 32 % 2, c = lane % kChunks, row = lane / kChunks % kRowsStore;
        // LDS row q holds its 16-byte chunk j at place j ^ turn(q), so that 16 rows' chunks j are in different banks.
        // Rows and places are different bits of an address: one exclusive or goes from one to the next.
        auto turn = [](uint32_t q) { return q / (256 / kRow) % kChunks; };
        uint8_t* mine = lds + (WALK ? S * C::kStage : 0) + wave * 32 * kRow;
        const uint32_t mine0 = (uint32_t)(mine - lds);
        const uint32_t to0 = mine0 + r * kRow + ((4 * h * kEs / 16) ^ turn(r)) * 16 + 4 * h * kEs % 16;
        const uint32_t from0 = mine0 + row * kRow + (c ^ turn(row)) * 16;
        auto from = [&](int i) { return lds + ((from0 ^ (turn(i * kRowsStore) * 16)) + i * kRowsStore * kRow); };
        const Gemm4Args b = args_again();
        if constexpr (WALK) tile = tiles.at(b, number);
        const int64_t pitch = (OUT == kSums ? (int64_t)sums_pitch(b.N) : b.ld_y) * kEs;
        const bool full = tile.rows_m == BM && tile.rows_n == BN;
        uint8_t* out = reinterpret_cast<uint8_t*>(OUT == kSums ? b.work : b.y);
        if (OUT == kSums) out += (int64_t)tile.split * b.M * pitch;
        uint8_t* y = out + ((int64_t)tile.m0 + wm * C::kRowsM) * pitch + ((int64_t)tile.n0 + wn * C::kRowsN) * kEs;
        uint8_t* y_lane = y + row * pitch + c * 16;
        // Of a whole tile, a part is stored only when the next one has been written to LDS: the reads of a part are then
        // done, and LDS keeps a wavefront's reads before its later writes.
        constexpr int kParts = TM * TN / kPartN;
        u32x4 held[kStores];
        auto store = [&](int part) {
            const int m = part / (TN / kPartN), n0 = part % (TN / kPartN) * kPartN;
            uint8_t* to = y_lane + m * 32 * pitch + n0 * 32 * kEs;
            asm volatile("" : "+v"(to));   // formed here: kept for every store of a tile, addresses need scratch memory
#pragma unroll
            for (int i = 0; i < kStores; ++i, to += kRowsStore * pitch)
                if constexpr (OUT == kSums)   // which the join reads next
                    *reinterpret_cast<Out16*>(to) = Out16{{held[i][0], held[i][1], held[i][2], held[i][3]}};
                else   // streaming: the operands that other tiles read stay in the cache
                    __builtin_nontemporal_store(held[i], reinterpret_cast<Stream16*>(to));
        };
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            const int m = part / (TN / kPartN), n0 = part % (TN / kPartN) * kPartN;
            // (the compiler would convert everything before the first store, which needs scratch memory)
#pragma unroll
            for (int n = 0; n < kPartN; ++n) asm volatile("" : "+a"(acc[n0 + n][m]) : : "memory");
#pragma unroll
            for (int n = 0; n < kPartN; ++n)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint8_t* p = lds + (to0 ^ ((n * 32 + 8 * g) * kEs));
                    const f32x16& v = acc[n0 + n][m];
                    if constexpr (OUT == kBf16)
                        *reinterpret_cast<uint2*>(p) =
                            make_uint2(bf16_pair(v[4 * g], v[4 * g + 1]), bf16_pair(v[4 * g + 2], v[4 * g + 3]));
                    else
                        *reinterpret_cast<float4*>(p) = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
                }
            if (full) {
                if (part > 0) store(part - 1);
#pragma unroll
                for (int i = 0; i < kStores; ++i)
                    held[i] = *reinterpret_cast<const u32x4*>(from(i));
                if (part + 1 == kParts) store(part);
            } else {
#pragma unroll 1
                for (int i = 0; i < kStores; ++i) {
                    const int left_m = tile.rows_m - wm * C::kRowsM - m * 32 - i * kRowsStore - (int)row;
                    const int left_n = tile.rows_n - wn * C::kRowsN - n0 * 32 - (int)c * (16 / kEs);
                    const uint8_t* p = from(i);
                    uint8_t* to = y_lane + (m * 32 + i * kRowsStore) * pitch + n0 * 32 * kEs;
                    if (left_m <= 0 || left_n <= 0) continue;
                    if (left_n >= 16 / kEs) {
                        *reinterpret_cast<Out16*>(to) = *reinterpret_cast<const Out16*>(p);
                    } else {
                        for (int e = 0; e < left_n; ++e) {
                            if constexpr (OUT == kBf16)
                                reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(p)[e];
                            else
                                reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(p)[e];
                        }
                    }
                }
            }
        }
        if constexpr (!WALK) return;
        stored = full;
        number += gridDim.x;
        if (number >= tiles.count) return;
    }
}

// Adds the sums of the parts of k, in their order: 4 columns of a row a thread.
template <bool BF>
__global__ __launch_bounds__(256) void k_gemm4_join(Gemm4Args a, int splits) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const int pitch = sums_pitch(a.N), quads = (a.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / quads;
    const int n = (int)(i % quads) * 4;
    if (m >= a.M) return;
    const float* p = reinterpret_cast<const float*>(a.work) + m * pitch + n;
    f32x4 c = *reinterpret_cast<const f32x4*>(p);
    int s = 1;
    for (; s + 3 <= splits; s += 3) {   // three loads under way at a time
        f32x4 v[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) v[u] = *reinterpret_cast<const f32x4*>(p + (int64_t)(s + u) * a.M * pitch);
#pragma unroll
        for (int u = 0; u < 3; ++u) c += v[u];
    }
    for (; s < splits; ++s) c += *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.M * pitch);
    if constexpr (BF) {
        uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * a.ld_y + n;
        const Out8 o = {{bf16_pair(c[0], c[1]), bf16_pair(c[2], c[3])}};
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
            if (n + e < a.N) y[e] = c[e];
    }
}

template <int BM, int BN, int WM, int S, int SP, int OUT, bool GROUPED>
hipError_t launch_tile_kernel(const Gemm4Args& a, int tiles_m, int tiles_n, int splits, hipStream_t st) {
    using C = TileCfg<BM, BN, WM, S, SP>;
    // the walk's output goes through LDS of its own (4 KiB a wavefront)
    constexpr int kOut = 16384;
    constexpr bool WALK = BM * BN == 256 * 256;
    constexpr int kLds = C::kLds + (WALK ? kOut : 0);
    auto kernel = k_gemm4<BM, BN, WM, S, SP, OUT, GROUPED, WALK>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_big_lds(kernel, kLds, done);
    if (e != hipSuccess) return e;
    const int count = tiles_m * tiles_n * splits;
    return launch_kernel(kernel, dim3((unsigned)(WALK && count > kCus ? kCus : count)), 256, kLds, st, a, tiles_m, tiles_n,
                         splits);
}

template <int BM, int BN, int WM, int S, int SP>
hipError_t launch_tiles(const Gemm4Args& a, hipStream_t st) {
    const int tiles_m = (int)(((int64_t)a.M + BM - 1) / BM), tiles_n = (int)(((int64_t)a.N + BN - 1) / BN);
    return a.y_bf16 ? launch_tile_kernel<BM, BN, WM, S, SP, kBf16, false>(a, tiles_m, tiles_n, 1, st)
                    : launch_tile_kernel<BM, BN, WM, S, SP, kF32, false>(a, tiles_m, tiles_n, 1, st);
}

// The same, or with k in parts and their join.
template <int BM, int BN, int WM, int S, int SP>
hipError_t launch_tiles_or_parts(const Gemm4Args& a, int splits, hipStream_t st) {
    if (splits == 1) return launch_tiles<BM, BN, WM, S, SP>(a, st);
    const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN;
    const hipError_t e = launch_tile_kernel<BM, BN, WM, S, SP, kSums, false>(a, tiles_m, tiles_n, splits, st);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(((int64_t)a.M * ((a.N + 3) / 4) + 255) / 256));
    return launch_kernel(a.y_bf16 ? k_gemm4_join<true> : k_gemm4_join<false>, grid, 256, 0, st, a, splits);
}

template <int BM, int BN, int WM, int S, int SP>
hipError_t launch_group_tiles(const Gemm4Args& a, hipStream_t st) {
    const int tiles_m = (int)group_tiles(a.M, a.experts, BM), tiles_n = (int)(((int64_t)a.N + BN - 1) / BN);
    return a.y_bf16 ? launch_tile_kernel<BM, BN, WM, S, SP, kBf16, true>(a, tiles_m, tiles_n, 1, st)
                    : launch_tile_kernel<BM, BN, WM, S, SP, kF32, true>(a, tiles_m, tiles_n, 1, st);
}

// Few activation rows: bound by the one read of the weights (1 x 5120 x 5120: 4.6 us, 3.0 TB/s with a launch in it; 1 x
// 13824 x 5120: 7.9, 4.8 TB/s; 96 rows in 32 groups, 4096 x 4096: 58, 4.9 TB/s).  A ring of 2 units, 4 wavefronts: with 3
// units a workgroup fewer fits a compute unit (10% longer in groups), with 8 wavefronts the same (20%).  A workgroup has
// up to 32 weight rows and W wavefronts that split k between them.  Each wavefront runs on its own: it loads a group of
// columns of all rows (a unit) at a time into its own ring of S units in LDS (XL loads of 8 activation rows, 4 of weight
// rows, and the scales of 32 rows of either), and waits for nothing but its own loads.
template <int W, int S, int XL>
struct ThinCfg {
    static constexpr int kLoads = 6 + XL;
    static constexpr int kAtX = 4096 + 256, kAtXScales = kAtX + XL * 1024, kUnit = kAtXScales + 256;
    static constexpr int kRing = W * S * kUnit, kPart = W * 4096, kLds = kRing > kPart ? kRing : kPart;
};

template <int W, int S, int XL, int OUT, bool GROUPED>
__global__ __launch_bounds__(W * kWave) void k_gemm4_thin(Gemm4Args a, int rows, int tiles_m, int tiles_n) {
    using C = ThinCfg<W, S, XL>;
    constexpr int kLoads = C::kLoads, kUnit = C::kUnit;
    // vmcnt counts to 63; activation rows are one block of 32, or a part of one
    static_assert(S * kLoads < 64 && XL <= 4);
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Tile tile{0, a.M, (int)blockIdx.x * rows, 0, 0, 0};
    if constexpr (GROUPED) {   // (`rows` is 32)
        Tiles<XL * 8, 32, true> tiles(a, tiles_m, tiles_n, 1);
        if ((int)blockIdx.x >= tiles.count) return;
        tile = tiles.at(a, blockIdx.x);
    }
    const int m0 = tile.m0, rows_m = tile.rows_m, expert = tile.expert, n0 = tile.n0;
    const int rows_n = a.N - n0 < rows ? a.N - n0 : rows;
    const int u0 = a.groups * wave / W, u1 = a.groups * (wave + 1) / W;
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds + wave * S * kUnit;
    const uint8_t* ring_p = lds + wave * S * kUnit;
    const bool indexed = GROUPED && a.index;
    auto x_row = [&](int r, bool& none) {
        const int row = a.index[m0 + (r < rows_m ? r : 0)];
        none = r >= rows_m || row < 0 || row >= a.x_rows;
        return row;
    };
    uint32_t voff_w[4], voff_x[XL], voff_we, voff_xe;   // the layout of a stage of a tile
    voff_we = (uint32_t)lane * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 8;
        voff_w[i] = (uint32_t)r * (uint32_t)a.ld_w + (uint32_t)((lane % 8) ^ (r / 2 % 8)) * 16;
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = i * 8 + lane / 8;
        int row = r;
        bool none = false;
        if (indexed) row = x_row(row, none);
        voff_x[i] = none ? kFar : (uint32_t)row * (uint32_t)a.ld_x + (uint32_t)((lane % 8) ^ (r / 2 % 8)) * 16;
    }
    {
        uint32_t row = (uint32_t)lane / 2;
        bool none = false;
        if (indexed) row = x_row(row, none);
        voff_xe = none ? kFar : row * 8 + (uint32_t)lane % 2 * 4;
    }
    const int64_t at_m = indexed ? 0 : m0;
    const uint64_t base_x = (uint64_t)(a.xq + at_m * a.ld_x), base_xe = (uint64_t)(a.xe + at_m * 8);
    const uint64_t base_w = (uint64_t)(a.wq + (GROUPED ? expert * a.ld_wexpert : 0) + n0 * a.ld_w);
    const uint64_t base_we = (uint64_t)(a.we + (GROUPED ? expert * a.ld_weexpert : 0) + n0 * 8ll);
    const int64_t have_x = indexed ? a.x_rows : rows_m;
    const uint32_t stride = (uint32_t)a.groups * kGroupBytes;
    const uint32_t size_x = have_x ? (uint32_t)((have_x - 1) * a.ld_x) + stride : 0;
    const uint32_t size_w = (uint32_t)((rows_n - 1) * a.ld_w) + stride;
    auto load = [&](int u, int slot) {   // past the wavefront's part: from empty buffers
        const bool in = u < u1;
        const uint32_t at = (uint32_t)u * kGroupBytes;
        const u32x4 rw = rsrc_of(base_w + at, in ? size_w - at : 0);
        const u32x4 rx = rsrc_of(base_x + at, in && size_x ? size_x - at : 0);
        const u32x4 rwe = rsrc_of(base_we + u * a.ld_we, in ? (uint32_t)rows_n * 8 : 0);
        const u32x4 rxe = rsrc_of(base_xe + u * a.ld_xe, in ? (uint32_t)have_x * 8 : 0);
        asm volatile("s_nop 4" ::"s"(rw), "s"(rx), "s"(rwe), "s"(rxe));
        const uint32_t to = ring + slot * kUnit;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_lds16(rw, voff_w[i], to + i * 1024);
        load_lds4(rwe, voff_we, to + 4096);
#pragma unroll
        for (int i = 0; i < XL; ++i) load_lds16(rx, voff_x[i], to + C::kAtX + i * 1024);
        load_lds4(rxe, voff_xe, to + C::kAtXScales);
    };
#pragma unroll
    for (int s = 0; s < S; ++s) load(u0 + s, s);
    // with fewer than 32 rows of activations in the ring, columns past them repeat its first rows
    constexpr int kWrap = XL < 4 ? XL * 8 : 32;
    uint32_t col_w[4], col_x[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        const int r = lane % kWrap;
        col_w[ks] = (lane % 32) * kGroupBytes + ((ks + lane / 32 * 4) ^ (lane / 2 % 8)) * 16;
        col_x[ks] = r * kGroupBytes + ((ks + lane / 32 * 4) ^ (r / 2 % 8)) * 16;
    }
    const uint32_t at_we = 4096 + lane % 32 * 8 + lane / 32 * 4;
    const uint32_t at_xe = C::kAtXScales + lane % kWrap * 8 + lane / 32 * 4;
    f32x16 acc = (f32x16)(0.0f);
    int slot = 0;
    for (int u = u0; u < u1; ++u) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * kLoads) : "memory");
        const uint8_t* p = ring_p + slot * kUnit;
        i32x4 fw[4], fx[4];
        const int sw = *reinterpret_cast<const int*>(p + at_we), sx = *reinterpret_cast<const int*>(p + at_xe);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            fw[ks] = *reinterpret_cast<const i32x4*>(p + col_w[ks]);
            fx[ks] = *reinterpret_cast<const i32x4*>(p + C::kAtX + col_x[ks]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: refill it
        load(u + S, slot);
        static_for<4>([&](auto ks) { acc = mfma4<ks>(fw[ks], fx[ks], acc, sw, sx); });
        slot = slot + 1 < S ? slot + 1 : 0;
    }
    wait_stage<0>();
    float* part = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < 16; ++i) part[(wave * 16 + i) * kWave + lane] = acc[i];
    __syncthreads();
    const int most = rows_m < XL * 8 ? rows_m : XL * 8;
    for (int o = threadIdx.x; o < most * 32; o += W * kWave) {
        const int m = o / 32, n = o % 32;
        if (n >= rows_n) continue;
        const float* p = part + (n / 8 * 4 + n % 4) * kWave + n / 4 % 2 * 32 + m % 32;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) y += p[w * 16 * kWave];
        const int64_t at = (int64_t)(m0 + m) * a.ld_y + n0 + n;
        if constexpr (OUT == kBf16)
            reinterpret_cast<uint16_t*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)y);
        else
            reinterpret_cast<float*>(a.y)[at] = y;
    }
}

// (of rows in groups, 32 weight rows a workgroup)
template <int W, int S, int XL, int OUT, bool GROUPED>
hipError_t launch_thin_kernel(const Gemm4Args& a, int rows, hipStream_t st) {
    using C = ThinCfg<W, S, XL>;
    const int tiles_n = (a.N + rows - 1) / rows, tiles_m = GROUPED ? (int)group_tiles(a.M, a.experts, XL * 8) : 1;
    auto kernel = k_gemm4_thin<W, S, XL, OUT, GROUPED>;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_big_lds(kernel, C::kLds, done);
    if (e != hipSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)(tiles_n * tiles_m)), W * kWave, C::kLds, st, a, rows, tiles_m, tiles_n);
}

template <int OUT>
hipError_t launch_thin(const Gemm4Args& a, hipStream_t st) {
    const int rows = thin_rows(a.N);
    if (a.M <= 8) return launch_thin_kernel<4, 2, 1, OUT, false>(a, rows, st);
    if (a.M <= 16) return launch_thin_kernel<4, 2, 2, OUT, false>(a, rows, st);
    return launch_thin_kernel<4, 2, 4, OUT, false>(a, rows, st);
}

// 8 XL rows of a group at a time.
template <int XL>
hipError_t launch_group_thin(const Gemm4Args& a, hipStream_t st) {
    return a.y_bf16 ? launch_thin_kernel<4, 2, XL, kBf16, true>(a, 32, st)
                    : launch_thin_kernel<4, 2, XL, kF32, true>(a, 32, st);
}

}  // namespace

size_t gemm4_workspace(int M, int N, int groups) {
    if (M == 0 || N == 0) return 0;
    const Plan4 p = plan4(M, N, groups);
    return p.splits > 1 ? (size_t)p.splits * M * sums_pitch(N) * 4 : 0;
}

hipError_t launch_gemm4(const Gemm4Args& a, hipStream_t st) {
    const Plan4 p = plan4(a.M, a.N, a.groups);
    switch (p.tile) {
    case 0: return launch_tiles<256, 256, 2, 2, 48>(a, st);
    case 1: return launch_tiles_or_parts<128, 256, 2, 3, 32>(a, p.splits, st);
    case 2: return launch_tiles_or_parts<128, 128, 2, 3, 16>(a, p.splits, st);
    case 3: return launch_tiles_or_parts<64, 256, 1, 3, 16>(a, p.splits, st);
    case 4: return launch_tiles_or_parts<32, 256, 1, 4, 8>(a, p.splits, st);
    case 5: return launch_tiles_or_parts<64, 64, 2, 4, 4>(a, p.splits, st);
    default: return a.y_bf16 ? launch_thin<kBf16>(a, st) : launch_thin<kF32>(a, st);
    }
}

hipError_t launch_gemm4_grouped(const Gemm4Args& a, hipStream_t st) {
    switch (plan4_grouped(a.M, a.experts, a.N, a.groups)) {
    case 0: return launch_group_tiles<256, 256, 2, 2, 48>(a, st);
    case 1: return launch_group_tiles<128, 256, 2, 3, 32>(a, st);
    case 3: return launch_group_tiles<64, 256, 1, 3, 16>(a, st);
    case 4: return launch_group_tiles<32, 256, 1, 4, 8>(a, st);
    case kThin4: return launch_group_thin<1>(a, st);
    default: return launch_group_thin<2>(a, st);
    }
}

}  // namespace qamw
