// C ABI of the 8-bit linear layers (declared in include/qamw_w8.h).  Every argument is checked here, in
// host code, before anything is queued; then the kernels are launched on the caller's stream.
#include <cmath>

#include "qamw_w8.h"
#include "qamw_w8_launch.hpp"

using namespace qamw;

namespace {

// sizes of the product that the kernels take
bool gemm8_fits(int32_t M, int32_t d_out, int32_t d_in) {
    return M <= QAMW_GEMM8_MAX_ROWS && d_out <= QAMW_GEMM8_MAX_ROWS && d_in <= QAMW_GEMM8_MAX_COLS &&
           (int64_t)M * d_out <= QAMW_GEMM8_MAX_OUT;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int hip_rc(hipError_t e) { return e == hipSuccess ? QAMW_OK : QAMW_ERR_HIP; }

bool is_dtype(qamw_dtype t) { return t == QAMW_F32 || t == QAMW_BF16; }

uintptr_t elem_bytes(qamw_dtype t) { return t == QAMW_BF16 ? 2 : 4; }

// rows x d, as both row operators limit them
int check_rows(int32_t rows, int32_t d) {
    if (rows < 0 || d < 1) return QAMW_ERR_ARG;
    if (rows > QAMW_MAX_ROWS || d > QAMW_W8_MAX_COLS) return QAMW_ERR_UNSUPPORTED;
    return QAMW_OK;
}

// a code matrix: 16-byte rows
bool codes_ok(const int8_t* q, int64_t ld, int32_t d) { return q && aligned(q, 16) && ld >= d && ld % 16 == 0; }

}  // namespace

extern "C" {

size_t qamw_q8_stride(int32_t d) { return d <= 0 ? 0 : ((size_t)d + 15) / 16 * 16; }

int qamw_quant8(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_gate,
                int64_t ld_gate, const float* d_scale, int8_t* d_q, int64_t ld_q, float* d_row_scale,
                int32_t* d_status, void* stream) {
    if (!is_dtype(x_dtype)) return QAMW_ERR_ARG;
    const int rc = check_rows(rows, d);
    if (rc) return rc;
    if (ld_x < d || (d_gate && ld_gate < d)) return QAMW_ERR_ARG;
    if (rows == 0) return QAMW_OK;
    const uintptr_t e = elem_bytes(x_dtype);
    if (!d_x || !d_row_scale || !aligned(d_x, e) || !aligned(d_gate, e) || !aligned(d_scale, 4) ||
        !aligned(d_row_scale, 4) || !aligned(d_status, 4) || !codes_ok(d_q, ld_q, d))
        return QAMW_ERR_ARG;
    Rows8Args a{};
    a.x = d_x;
    a.x_bf16 = x_dtype == QAMW_BF16;
    a.rows = rows;
    a.d = d;
    a.ld_x = ld_x;
    a.other = d_gate;
    a.ld_other = ld_gate;
    a.factor = d_scale;
    a.q = d_q;
    a.ld_q = ld_q;
    a.row_scale = d_row_scale;
    a.status = d_status;
    return hip_rc(launch_quant8(a, (hipStream_t)stream));
}

int qamw_dequant8(const int8_t* d_q, int32_t rows, int32_t d, int64_t ld_q, const float* d_row_scale,
                  const float* d_scale, void* d_out, qamw_dtype out_dtype, int64_t ld_out, void* stream) {
    if (!is_dtype(out_dtype) || rows < 0 || d < 1 || ld_out < d) return QAMW_ERR_ARG;
    if (rows > QAMW_MAX_ROWS || d > QAMW_MAX_ROWS) return QAMW_ERR_UNSUPPORTED;
    if (rows == 0) return QAMW_OK;
    if (!codes_ok(d_q, ld_q, d) || !d_row_scale || !d_out || !aligned(d_row_scale, 4) || !aligned(d_scale, 4) ||
        !aligned(d_out, elem_bytes(out_dtype)))
        return QAMW_ERR_ARG;
    Dequant8Args a{};
    a.q = d_q;
    a.rows = rows;
    a.d = d;
    a.ld_q = ld_q;
    a.row_scale = d_row_scale;
    a.scale = d_scale;
    a.out = d_out;
    a.out_bf16 = out_dtype == QAMW_BF16;
    a.ld_out = ld_out;
    return hip_rc(launch_dequant8(a, (hipStream_t)stream));
}

int qamw_rmsnorm8(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_residual,
                  int64_t ld_res, const float* d_weight, float eps, void* d_sum, int64_t ld_sum, int8_t* d_q,
                  int64_t ld_q, float* d_row_scale, int32_t* d_status, void* stream) {
    if (!is_dtype(x_dtype)) return QAMW_ERR_ARG;
    const int rc = check_rows(rows, d);
    if (rc) return rc;
    if (ld_x < d || (d_residual && ld_res < d) || (d_sum && ld_sum < d)) return QAMW_ERR_ARG;
    if (!std::isfinite(eps) || eps < 0.0f) return QAMW_ERR_ARG;
    if (rows == 0) return QAMW_OK;
    const uintptr_t e = elem_bytes(x_dtype);
    if (!d_x || !d_row_scale || !aligned(d_x, e) || !aligned(d_residual, e) || !aligned(d_sum, e) ||
        !aligned(d_weight, 4) || !aligned(d_row_scale, 4) || !aligned(d_status, 4) || !codes_ok(d_q, ld_q, d))
        return QAMW_ERR_ARG;
    // h is written in place over an input only element by element
    if ((d_sum == d_x && ld_sum != ld_x) || (d_sum && d_sum == d_residual && ld_sum != ld_res)) return QAMW_ERR_ARG;
    Rows8Args a{};
    a.x = d_x;
    a.x_bf16 = x_dtype == QAMW_BF16;
    a.rows = rows;
    a.d = d;
    a.ld_x = ld_x;
    a.other = d_residual;
    a.ld_other = ld_res;
    a.factor = d_weight;
    a.eps = (double)eps;
    a.sum = d_sum;
    a.ld_sum = ld_sum;
    a.q = d_q;
    a.ld_q = ld_q;
    a.row_scale = d_row_scale;
    a.status = d_status;
    return hip_rc(launch_rmsnorm8(a, (hipStream_t)stream));
}

size_t qamw_gemm8_workspace(int32_t M, int32_t d_out, int32_t d_in) {
    if (M < 0 || d_out < 0 || d_in < 1 || !gemm8_fits(M, d_out, d_in)) return 0;
    return gemm8_workspace(M, d_out, d_in);
}

int qamw_gemm8(const int8_t* d_xq, int64_t ld_x, const float* d_xs, int32_t M, const int8_t* d_wq, int64_t ld_w,
               const float* d_wscale, int32_t d_out, int32_t d_in, void* d_y, qamw_dtype y_dtype, int64_t ld_y,
               void* d_ws, size_t ws_bytes, void* stream) {
    if (!is_dtype(y_dtype) || M < 0 || d_out < 0 || d_in < 1 || ld_y < d_out) return QAMW_ERR_ARG;
    if (!gemm8_fits(M, d_out, d_in) || ld_x > QAMW_GEMM8_MAX_LD || ld_w > QAMW_GEMM8_MAX_LD)
        return QAMW_ERR_UNSUPPORTED;
    if (M == 0 || d_out == 0) return QAMW_OK;
    if (!codes_ok(d_xq, ld_x, d_in) || !codes_ok(d_wq, ld_w, d_in) || !d_xs || !d_wscale || !d_y ||
        !aligned(d_xs, 4) || !aligned(d_wscale, 4) || !aligned(d_y, elem_bytes(y_dtype)))
        return QAMW_ERR_ARG;
    const size_t need = gemm8_workspace(M, d_out, d_in);
    if (need && (!d_ws || !aligned(d_ws, 256) || ws_bytes < need)) return QAMW_ERR_WORKSPACE;
    Gemm8Args a{};
    a.xq = d_xq;
    a.ld_x = ld_x;
    a.xs = d_xs;
    a.M = M;
    a.wq = d_wq;
    a.ld_w = ld_w;
    a.ws = d_wscale;
    a.N = d_out;
    a.K = d_in;
    a.y = d_y;
    a.y_bf16 = y_dtype == QAMW_BF16;
    a.ld_y = ld_y;
    a.work = d_ws;
    return hip_rc(launch_gemm8(a, (hipStream_t)stream));
}

}  // extern "C"
