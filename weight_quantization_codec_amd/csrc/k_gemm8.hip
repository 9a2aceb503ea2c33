// Product of 8-bit matrices: y[m][n] = xs_m ws_n sum_k xq[m][k] wq[n][k], exact 32-bit integer sums on
// the matrix cores (v_mfma_i32_32x32x32_i8).
//
// Both operands have their columns k contiguous.  An operand of the instruction is 16 consecutive bytes
// of one row a lane; which k a byte belongs to does not matter as long as both operands agree, so the
// rows are used as they are stored.
#include "qamw_device.hpp"
#include "qamw_w8_launch.hpp"

namespace qamw {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;   // bytes of k a step: one cache line of every row of a tile

// 16 bytes of output at any alignment of its elements
struct __attribute__((packed, aligned(2))) Out16 {
    uint32_t w[4];
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

// Waits until at most N of the wavefront's loads and none of its LDS reads are under way, then for the
// workgroup.
template <int N>
__device__ __forceinline__ void wait_stage() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A tile of BM activation rows by BN weight rows, 2 x 2 wavefronts, S stages of kStep bytes of k in LDS.
template <int BM, int BN, int S>
struct TileCfg {
    static constexpr int kTM = BM / 64, kTN = BN / 64;       // 32 x 32 blocks of a wavefront
    static constexpr int kLoads = (BM + BN) / 32;            // loads of a wavefront and stage (8 rows each)
    static constexpr int kStage = (BM + BN) * kStep;         // bytes
    static constexpr int kLds = S * kStage;
};

// The workgroup's tile.  Workgroups go round the 8 XCDs; each XCD gets a contiguous run of tiles, taken
// kGroup tile rows at a time, so that the tiles an XCD works on at once share rows in its L2.
constexpr int kXcds = 8, kGroup = 8;
__device__ __forceinline__ void tile_of(int b, int tiles, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int per = tiles / kXcds, rest = tiles % kXcds, x = b % kXcds;
    const int t = x * per + (x < rest ? x : rest) + b / kXcds;
    const int group = t / (kGroup * tiles_n), first = group * kGroup;
    const int in = tiles_m - first < kGroup ? tiles_m - first : kGroup, at = t - first * tiles_n;
    tm = first + at % in;
    tn = at / in;
}

template <int BM, int BN, int S, bool BF>
__global__ __launch_bounds__(256, 1) void k_gemm8(Gemm8Args a, int tiles_m, int tiles_n) {
    using C = TileCfg<BM, BN, S>;
    constexpr int TM = C::kTM, TN = C::kTN;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    int tile_m, tile_n;
    tile_of(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * BM, n0 = (int64_t)tile_n * BN;
    const int rows_m = a.M - tile_m * BM < BM ? a.M - tile_m * BM : BM;
    const int rows_n = a.N - tile_n * BN < BN ? a.N - tile_n * BN : BN;
    const int steps = (a.K + kStep - 1) / kStep, pad_k = (a.K + 15) / 16 * 16;

    // Loads.  One moves 8 rows of 128 bytes; LDS row r holds its 16-byte chunk c at place c ^ (r % 8), so
    // that the 8 lanes of a read phase, at one c of 8 rows, touch all banks once.  Rows past the matrix
    // repeat its last row (their sums are not stored).
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    uint32_t voff[C::kLoads];
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
        const bool is_x = i < BM / 32;
        int row = ((is_x ? i : i - BM / 32) * 4 + wave) * 8 + lane / 8;
        const int last = (is_x ? rows_m : rows_n) - 1;
        row = row < last ? row : last;
        voff[i] = (uint32_t)row * (uint32_t)(is_x ? a.ld_x : a.ld_w) + (uint32_t)((lane % 8) ^ (lane / 8)) * 16;
    }
    const uint64_t base_x = (uint64_t)(a.xq + m0 * a.ld_x), base_w = (uint64_t)(a.wq + n0 * a.ld_w);
    const uint32_t size_x = (uint32_t)((rows_m - 1) * a.ld_x) + pad_k, size_w = (uint32_t)((rows_n - 1) * a.ld_w) + pad_k;
    // The buffers of step t: they end with the last row, and are empty past the last step (such loads
    // touch no memory, and keep the count of loads under way the same in every step).
    auto rsrc = [&](uint64_t base, uint32_t size, int t) {
        const uint64_t p = base + (uint64_t)t * kStep;
        u32x4 r;
        r[0] = __builtin_amdgcn_readfirstlane((uint32_t)p);
        r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32) & 0xFFFFu);
        r[2] = __builtin_amdgcn_readfirstlane(t < steps ? size - (uint32_t)t * kStep : 0u);
        r[3] = 0x00020000u;
        return r;
    };
    auto load = [&](int i, u32x4 rx, u32x4 rw, uint32_t stage) {
        const bool is_x = i < BM / 32;
        load_lds16(is_x ? rx : rw, voff[i], stage + (uint32_t)(i * 4 + wave) * 1024);
    };
    // Bytes past K of the last step's activations become zeros.
    auto clear_tail = [&](uint8_t* st) {
        const int at = a.K % kStep;
        for (int i = threadIdx.x; i < BM * (kStep - at); i += 256) {
            const int row = i / (kStep - at), k = at + i % (kStep - at);
            st[row * kStep + ((k / 16) ^ (row % 8)) * 16 + k % 16] = 0;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    const bool tail = a.K % kStep != 0;

    // Operands: block row lane % 32, 16-byte chunk 2 ks + lane / 32 of sub-step ks.
    const int wm = wave / 2, wn = wave % 2;
    uint32_t col[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) col[ks] = (lane % 32) * kStep + (((2 * ks + lane / 32) ^ (lane % 8)) * 16);
    const uint32_t row_x = wm * (BM / 2) * kStep, row_w = (BM + wn * (BN / 2)) * kStep;
    i32x4 fx[2][TM], fw[2][TN];
    auto read = [&](int i, int set, const uint8_t* st, int ks) {
        if (i < TN)
            fw[set][i] = *reinterpret_cast<const i32x4*>(st + row_w + i * 32 * kStep + col[ks]);
        else
            fx[set][i - TN] = *reinterpret_cast<const i32x4*>(st + row_x + (i - TN) * 32 * kStep + col[ks]);
    };
    i32x16 acc[TN][TM];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[n][m] = (i32x16)(0);

#pragma unroll
    for (int s = 0; s < S; ++s) {
        const u32x4 rx = rsrc(base_x, size_x, s), rw = rsrc(base_w, size_w, s);
        asm volatile("s_nop 4" ::"s"(rx), "s"(rw));
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) load(i, rx, rw, lds0 + s * C::kStage);
    }
    wait_stage<(S - 1) * C::kLoads>();
    if (steps == 1 && tail) clear_tail(lds);
#pragma unroll
    for (int i = 0; i < TM + TN; ++i) read(i, 0, lds, 0);

    int buf = 0;
    for (int t = 0; t < steps; ++t) {
        const int next = buf + 1 < S ? buf + 1 : 0;
        const uint8_t* cur_p = lds + buf * C::kStage;
        uint8_t* next_p = lds + next * C::kStage;
        u32x4 rx, rw;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            // sub-step ks multiplies set ks % 2 while the next set is read; the last one first waits for
            // the next stage, and refills this one, which every wavefront has then read
            if (ks == 3) {
                wait_stage<(S - 2) * C::kLoads>();
                if (tail && t + 2 == steps) clear_tail(next_p);
                rx = rsrc(base_x, size_x, t + S);
                rw = rsrc(base_w, size_w, t + S);
                // a scalar register written by a vector instruction needs five wait states before a load
                // reads it; the compiler does not look into the assembly of the loads
                asm volatile("s_nop 4" ::"s"(rx), "s"(rw));
            }
#pragma unroll
            for (int j = 0; j < TM * TN; ++j) {
                if (j < TM + TN) read(j, (ks + 1) % 2, ks == 3 ? next_p : cur_p, (ks + 1) % 4);
                if (ks == 3) {
#pragma unroll
                    for (int i = 0; i < C::kLoads; ++i)
                        if (i * TM * TN / C::kLoads == j) load(i, rx, rw, lds0 + buf * C::kStage);
                }
                const int n = j / TM, m = j % TM;
                acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[ks % 2][n], fx[ks % 2][m], acc[n][m], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        buf = next;
    }

    // Rows of y through LDS, 32 at a time and wavefront, for stores of whole lines.  A lane has column
    // m = lane % 32 of each block and rows n = 8 g + 4 (lane / 32) + 0..3.
    wait_stage<0>();
    constexpr int kEs = BF ? 2 : 4, kRow = BN / 2 * kEs, kChunks = kRow / 16;
    uint8_t* mine = lds + wave * 32 * kRow;
    const int64_t nw = n0 + wn * (BN / 2);
    float ws[TN][4][4];
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = nw + n * 32 + 8 * g + 4 * (lane / 32) + i;
                ws[n][g][i] = a.ws[at < a.N ? at : a.N - 1];
            }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        const int64_t mw = m0 + wm * (BM / 2) + m * 32;
        if (mw >= a.M) break;
        const int r = lane % 32;
        const float xs = a.xs[mw + r < a.M ? mw + r : a.M - 1];
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)acc[n][m][4 * g + i] * xs * ws[n][g][i];
                const int byte = (n * 32 + 8 * g + 4 * (lane / 32)) * kEs;
                uint8_t* p = mine + r * kRow + (((byte / 16) ^ r) % kChunks) * 16 + byte % 16;
                if constexpr (BF)
                    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
                else
                    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < 32 * kChunks / kWave; ++i) {
            const int row = (i * kWave + lane) / kChunks, c = (i * kWave + lane) % kChunks;
            const Out16 v = *reinterpret_cast<const Out16*>(mine + row * kRow + ((c ^ row) % kChunks) * 16);
            const int64_t mm = mw + row, nn = nw + c * (16 / kEs);
            if (mm >= a.M) continue;
            if constexpr (BF) {
                uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + mm * a.ld_y + nn;
                if (nn + 8 <= a.N) {
                    *reinterpret_cast<Out16*>(y) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (nn + e < a.N) y[e] = (uint16_t)(v.w[e / 2] >> (16 * (e % 2)));
                }
            } else {
                uint32_t* y = reinterpret_cast<uint32_t*>(a.y) + mm * a.ld_y + nn;
                if (nn + 4 <= a.N) {
                    *reinterpret_cast<Out16*>(y) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < a.N) y[e] = v.w[e];
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

template <typename K>
hipError_t allow_big_lds(K kernel, int bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int BM, int BN, int S>
hipError_t launch_tiles(const Gemm8Args& a, hipStream_t st) {
    using C = TileCfg<BM, BN, S>;
    const int64_t tiles_m = ((int64_t)a.M + BM - 1) / BM, tiles_n = ((int64_t)a.N + BN - 1) / BN;
    const int64_t slab = (1 << 22) / tiles_n;   // row tiles a launch: the grid stays below 2^32 work items
    for (int64_t m = 0; m < tiles_m; m += slab) {
        Gemm8Args s = a;
        const int64_t tiles = tiles_m - m < slab ? tiles_m - m : slab, rows = (int64_t)a.M - m * BM;
        s.xq += m * BM * a.ld_x;
        s.xs += m * BM;
        s.M = (int)(rows < tiles * BM ? rows : tiles * BM);
        s.y = reinterpret_cast<char*>(a.y) + m * BM * a.ld_y * (a.y_bf16 ? 2 : 4);
        const dim3 grid((unsigned)(tiles * tiles_n));
        hipError_t e;
        if (a.y_bf16) {
            e = allow_big_lds(k_gemm8<BM, BN, S, true>, C::kLds);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((k_gemm8<BM, BN, S, true>), grid, dim3(256), C::kLds, st, s, (int)tiles, (int)tiles_n);
        } else {
            e = allow_big_lds(k_gemm8<BM, BN, S, false>, C::kLds);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((k_gemm8<BM, BN, S, false>), grid, dim3(256), C::kLds, st, s, (int)tiles, (int)tiles_n);
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t gemm8_workspace(int, int, int) { return 0; }

hipError_t launch_gemm8(const Gemm8Args& a, hipStream_t st) {
    if (a.M > 256) return launch_tiles<256, 256, 2>(a, st);
    return launch_tiles<128, 128, 4>(a, st);
}

}  // namespace qamw
