// Rows of bf16 or fp32 values in chunks of 8 columns, as the row kernels load and store them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qamw_device.hpp"

namespace qamw {

constexpr int kChunk = 8;            // columns of a chunk

// 16 bytes at any address that the element type allows: gfx950 loads and stores wide at any alignment
struct __attribute__((packed, aligned(2))) Bytes16 {
    uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) Float8 {
    float v[8];
};

// Two values as bf16, rounded to nearest even, by one v_cvt_pk_bf16_f32 (converted one by one, a pair takes four
// instructions).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
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

// The larger of a magnitude and |v|; NaN if either is (v_maximum3_f32).
__device__ __forceinline__ float top_of(float top, float v) {
    return __builtin_elementwise_maximum(top, __builtin_fabsf(v));
}

}  // namespace qamw
