// Host-side launchers of the 4-bit row and product kernels.  Arguments are validated by the C ABI
// layer (qamw_mx4_api.hip) before any of these is called.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "qamw_w8_launch.hpp"   // launch_kernel

namespace qamw {

constexpr int kGroupCols = 256, kGroupBytes = 128;   // a group of columns: 8 blocks of 32

// Rows to codes (k_rows4.hip): plain, gated, or behind a norm.
struct Rows4Args {
    const void* x;
    int x_bf16;
    int rows, d;
    int64_t ld_x;
    const void* other;     // gate, or residual (may be null)
    int64_t ld_other;
    const float* factor;   // channel scale, or norm weight (may be null)
    double eps;
    void* sum;             // norm: h, rounded to x's type (may be null)
    int64_t ld_sum;
    uint8_t* q;
    int64_t ld_q;
    uint8_t* e;
    int64_t ld_e;
    int32_t* status;
};
struct Dequant4Args {
    const uint8_t* q;
    int rows, d;
    int64_t ld_q;
    const uint8_t* e;
    int64_t ld_e;
    const float* scale;    // may be null
    void* out;
    int out_bf16;
    int64_t ld_out;
};
hipError_t launch_quant4(const Rows4Args& a, hipStream_t st);
hipError_t launch_rmsnorm4(const Rows4Args& a, hipStream_t st);
hipError_t launch_dequant4(const Dequant4Args& a, hipStream_t st);

// The products (k_gemm4.hip).
struct Gemm4Args {
    const uint8_t* xq;
    int64_t ld_x;
    const uint8_t* xe;
    int64_t ld_xe;
    int M;                 // rows of y
    const uint8_t* wq;
    int64_t ld_w;
    const uint8_t* we;
    int64_t ld_we;
    int N, groups;
    void* y;
    int y_bf16;
    int64_t ld_y;
    void* work;
    // rows in groups
    const int32_t* offsets;   // experts + 1
    int experts;
    int64_t ld_wexpert, ld_weexpert;
    const int32_t* index;     // may be null
    int x_rows;
};
size_t gemm4_workspace(int M, int N, int groups);
hipError_t launch_gemm4(const Gemm4Args& a, hipStream_t st);
hipError_t launch_gemm4_grouped(const Gemm4Args& a, hipStream_t st);

}  // namespace qamw
