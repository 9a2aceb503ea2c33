// What the kernels of tiled products share: loads from memory straight into LDS and the waits for them, and which
// tile a workgroup has.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

namespace qamw {

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

typedef uint32_t Stream16 __attribute__((ext_vector_type(4), aligned(2)));   // the same, for streaming stores

struct __attribute__((packed, aligned(2))) Out8 {
    uint32_t w[2];
};

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

// Values from one row of a part's sums to the next.
__host__ __device__ constexpr int sums_pitch(int n) { return (n + 63) / 64 * 64; }

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

// Lets a kernel use more than the default 64 KiB of LDS on the current device; `done` has a bit for each
// device where that has been said.
template <typename K>
inline hipError_t allow_big_lds(K kernel, int bytes, std::atomic<uint64_t>& done) {
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

}  // namespace qamw
