// Host-side launchers of the 8-bit row and product kernels.  Arguments are validated by the C ABI
// layer (qamw_w8_api.hip) before any of these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qamw {

// Launches a kernel and gives that launch's own error.  (hipGetLastError would also give an error that an earlier
// call of the thread has left.)  An error that is given here is not left for others.
template <typename... P, typename... A>
hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, int block, size_t lds, hipStream_t st, A... args) {
    auto launch = [&](P... values) {
        void* p[] = {&values...};
        return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3((unsigned)block), p, lds, st);
    };
    const hipError_t e = launch(args...);
    if (e != hipSuccess) (void)hipGetLastError();
    return e;
}

// Rows to codes (k_rows8.hip): plain, gated, or behind a norm.
struct Rows8Args {
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
    int8_t* q;
    int64_t ld_q;
    float* row_scale;
    int32_t* status;
};
struct Dequant8Args {
    const int8_t* q;
    int rows, d;
    int64_t ld_q;
    const float* row_scale;
    const float* scale;    // may be null
    void* out;
    int out_bf16;
    int64_t ld_out;
};
hipError_t launch_quant8(const Rows8Args& a, hipStream_t st);
hipError_t launch_rmsnorm8(const Rows8Args& a, hipStream_t st);
hipError_t launch_dequant8(const Dequant8Args& a, hipStream_t st);

// The product (k_gemm8.hip).
struct Gemm8Args {
    const int8_t* xq;
    int64_t ld_x;
    const float* xs;
    int M;
    const int8_t* wq;
    int64_t ld_w;
    const float* ws;
    int N, K;
    void* y;
    int y_bf16;
    int64_t ld_y;
    void* work;
};
size_t gemm8_workspace(int M, int N, int K);
hipError_t launch_gemm8(const Gemm8Args& a, hipStream_t st);

}  // namespace qamw
