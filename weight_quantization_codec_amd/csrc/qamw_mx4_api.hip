// C ABI of the 4-bit linear layers (declared in include/qamw_mx4.h).  Every argument is checked here, in
// host code, before anything is queued; then the kernels are launched on the caller's stream.
#include <cmath>

#include "qamw_mx4.h"
#include "qamw_mx4_launch.hpp"

using namespace qamw;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int hip_rc(hipError_t e) { return e == hipSuccess ? QAMW_OK : QAMW_ERR_HIP; }

bool is_dtype(qamw_dtype t) { return t == QAMW_F32 || t == QAMW_BF16; }

uintptr_t elem_bytes(qamw_dtype t) { return t == QAMW_BF16 ? 2 : 4; }

int64_t stride_of(int64_t d) { return (d + kGroupCols - 1) / kGroupCols * kGroupBytes; }

// codes of rows of `stride` bytes, and their scales
bool codes_ok(const uint8_t* q, int64_t ld, int64_t stride) {
    return q && aligned(q, 16) && ld >= stride && ld % 16 == 0;
}
bool scales_ok(const uint8_t* e, int64_t ld, int64_t rows) { return e && aligned(e, 8) && ld >= 8 * rows && ld % 8 == 0; }

int check_rows(int32_t rows, int32_t d, int32_t most) {
    if (rows < 0 || d < 1) return QAMW_ERR_ARG;
    if (rows > QAMW_MAX_ROWS || d > most) return QAMW_ERR_UNSUPPORTED;
    return QAMW_OK;
}

// sizes of the products that the kernels take
bool gemm4_fits(int32_t M, int32_t d_out, int32_t groups) {
    return M <= QAMW_GEMM4_MAX_ROWS && d_out <= QAMW_GEMM4_MAX_ROWS && groups <= QAMW_MX4_MAX_COLS / kGroupCols &&
           (int64_t)M * d_out <= QAMW_GEMM4_MAX_OUT;
}

}  // namespace

extern "C" {

size_t qamw_mx4_stride(int32_t d) { return d <= 0 ? 0 : (size_t)stride_of(d); }

int32_t qamw_mx4_groups(int32_t d) { return d <= 0 ? 0 : (int32_t)(stride_of(d) / kGroupBytes); }

int qamw_quant4(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_gate,
                int64_t ld_gate, const float* d_scale, uint8_t* d_q, int64_t ld_q, uint8_t* d_e, int64_t ld_e,
                int32_t* d_status, void* stream) {
    if (!is_dtype(x_dtype)) return QAMW_ERR_ARG;
    const int rc = check_rows(rows, d, QAMW_MX4_MAX_COLS);
    if (rc) return rc;
    if (ld_x < d || (d_gate && ld_gate < d)) return QAMW_ERR_ARG;
    if (rows == 0) return QAMW_OK;
    const uintptr_t e = elem_bytes(x_dtype);
    if (!d_x || !aligned(d_x, e) || !aligned(d_gate, e) || !aligned(d_scale, 4) || !aligned(d_status, 4) ||
        !codes_ok(d_q, ld_q, stride_of(d)) || !scales_ok(d_e, ld_e, rows))
        return QAMW_ERR_ARG;
    Rows4Args a{};
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
    a.e = d_e;
    a.ld_e = ld_e;
    a.status = d_status;
    return hip_rc(launch_quant4(a, (hipStream_t)stream));
}

int qamw_dequant4(const uint8_t* d_q, int32_t rows, int32_t d, int64_t ld_q, const uint8_t* d_e, int64_t ld_e,
                  const float* d_scale, void* d_out, qamw_dtype out_dtype, int64_t ld_out, void* stream) {
    if (!is_dtype(out_dtype)) return QAMW_ERR_ARG;
    const int rc = check_rows(rows, d, QAMW_MX4_MAX_COLS);
    if (rc) return rc;
    if (ld_out < d) return QAMW_ERR_ARG;
    if (rows == 0) return QAMW_OK;
    if (!codes_ok(d_q, ld_q, stride_of(d)) || !scales_ok(d_e, ld_e, rows) || !d_out || !aligned(d_scale, 4) ||
        !aligned(d_out, elem_bytes(out_dtype)))
        return QAMW_ERR_ARG;
    Dequant4Args a{};
    a.q = d_q;
    a.rows = rows;
    a.d = d;
    a.ld_q = ld_q;
    a.e = d_e;
    a.ld_e = ld_e;
    a.scale = d_scale;
    a.out = d_out;
    a.out_bf16 = out_dtype == QAMW_BF16;
    a.ld_out = ld_out;
    return hip_rc(launch_dequant4(a, (hipStream_t)stream));
}

int qamw_rmsnorm4(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_residual,
                  int64_t ld_res, const float* d_weight, float eps, void* d_sum, int64_t ld_sum, uint8_t* d_q,
                  int64_t ld_q, uint8_t* d_e, int64_t ld_e, int32_t* d_status, void* stream) {
    if (!is_dtype(x_dtype)) return QAMW_ERR_ARG;
    const int rc = check_rows(rows, d, QAMW_MX4_MAX_NORM_COLS);
    if (rc) return rc;
    if (ld_x < d || (d_residual && ld_res < d) || (d_sum && ld_sum < d)) return QAMW_ERR_ARG;
    if (!std::isfinite(eps) || eps < 0.0f) return QAMW_ERR_ARG;
    if (rows == 0) return QAMW_OK;
    const uintptr_t e = elem_bytes(x_dtype);
    if (!d_x || !aligned(d_x, e) || !aligned(d_residual, e) || !aligned(d_sum, e) || !aligned(d_weight, 4) ||
        !aligned(d_status, 4) || !codes_ok(d_q, ld_q, stride_of(d)) || !scales_ok(d_e, ld_e, rows))
        return QAMW_ERR_ARG;
    // h is written in place over an input only element by element
    if ((d_sum == d_x && ld_sum != ld_x) || (d_sum && d_sum == d_residual && ld_sum != ld_res)) return QAMW_ERR_ARG;
    Rows4Args a{};
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
    a.e = d_e;
    a.ld_e = ld_e;
    a.status = d_status;
    return hip_rc(launch_rmsnorm4(a, (hipStream_t)stream));
}

size_t qamw_gemm4_workspace(int32_t M, int32_t d_out, int32_t groups) {
    if (M < 0 || d_out < 0 || groups < 1 || !gemm4_fits(M, d_out, groups)) return 0;
    return gemm4_workspace(M, d_out, groups);
}

int qamw_gemm4(const uint8_t* d_xq, int64_t ld_x, const uint8_t* d_xe, int64_t ld_xe, int32_t M, const uint8_t* d_wq,
               int64_t ld_w, const uint8_t* d_we, int64_t ld_we, int32_t d_out, int32_t groups, void* d_y,
               qamw_dtype y_dtype, int64_t ld_y, void* d_ws, size_t ws_bytes, void* stream) {
    if (!is_dtype(y_dtype) || M < 0 || d_out < 0 || groups < 1 || ld_y < d_out) return QAMW_ERR_ARG;
    if (!gemm4_fits(M, d_out, groups) || ld_x > QAMW_GEMM4_MAX_LD || ld_w > QAMW_GEMM4_MAX_LD)
        return QAMW_ERR_UNSUPPORTED;
    if (M == 0 || d_out == 0) return QAMW_OK;
    const int64_t stride = (int64_t)groups * kGroupBytes;
    if (!codes_ok(d_xq, ld_x, stride) || !codes_ok(d_wq, ld_w, stride) || !scales_ok(d_xe, ld_xe, M) ||
        !scales_ok(d_we, ld_we, d_out) || !d_y || !aligned(d_y, elem_bytes(y_dtype)))
        return QAMW_ERR_ARG;
    const size_t need = gemm4_workspace(M, d_out, groups);
    if (need && (!d_ws || !aligned(d_ws, 256) || ws_bytes < need)) return QAMW_ERR_WORKSPACE;
    Gemm4Args a{};
    a.xq = d_xq;
    a.ld_x = ld_x;
    a.xe = d_xe;
    a.ld_xe = ld_xe;
    a.M = M;
    a.wq = d_wq;
    a.ld_w = ld_w;
    a.we = d_we;
    a.ld_we = ld_we;
    a.N = d_out;
    a.groups = groups;
    a.y = d_y;
    a.y_bf16 = y_dtype == QAMW_BF16;
    a.ld_y = ld_y;
    a.work = d_ws;
    return hip_rc(launch_gemm4(a, (hipStream_t)stream));
}

int qamw_gemm4_grouped(const uint8_t* d_xq, int64_t ld_x, const uint8_t* d_xe, int64_t ld_xe, int32_t x_rows,
                       const int32_t* d_index, int32_t rows, const uint8_t* d_wq, int64_t ld_w, int64_t ld_wexpert,
                       const uint8_t* d_we, int64_t ld_we, int64_t ld_weexpert, const int32_t* d_offsets,
                       int32_t experts, int32_t d_out, int32_t groups, void* d_y, qamw_dtype y_dtype, int64_t ld_y,
                       void* stream) {
    if (!is_dtype(y_dtype) || rows < 0 || x_rows < 0 || d_out < 0 || groups < 1 || experts < 1 || ld_y < d_out)
        return QAMW_ERR_ARG;
    if (!gemm4_fits(rows, d_out, groups) || x_rows > QAMW_GEMM4_MAX_ROWS || ld_x > QAMW_GEMM4_MAX_LD ||
        ld_w > QAMW_GEMM4_MAX_LD || experts > QAMW_GEMM4_MAX_EXPERTS ||
        (int64_t)experts * d_out > QAMW_GEMM4_MAX_EXPERT_ROWS)
        return QAMW_ERR_UNSUPPORTED;
    if (d_index ? !aligned(d_index, 4) : x_rows < rows) return QAMW_ERR_ARG;
    if (rows == 0 || d_out == 0) return QAMW_OK;
    const int64_t stride = (int64_t)groups * kGroupBytes;
    // (no rows of x: only indexes that stand for zeros can be given, and nothing of x is read)
    if ((x_rows && (!codes_ok(d_xq, ld_x, stride) || !scales_ok(d_xe, ld_xe, x_rows))) ||
        !codes_ok(d_wq, ld_w, stride) || ld_wexpert < 0 || ld_wexpert % 16 || !scales_ok(d_we, ld_we, d_out) ||
        ld_weexpert < 0 || ld_weexpert % 8 || !d_offsets || !aligned(d_offsets, 4) || !d_y ||
        !aligned(d_y, elem_bytes(y_dtype)))
        return QAMW_ERR_ARG;
    if (d_index && (int64_t)x_rows * ld_x > QAMW_GEMM4_MAX_INDEXED) return QAMW_ERR_UNSUPPORTED;
    Gemm4Args a{};
    a.xq = d_xq;
    a.ld_x = ld_x;
    a.xe = d_xe;
    a.ld_xe = ld_xe;
    a.M = rows;
    a.wq = d_wq;
    a.ld_w = ld_w;
    a.we = d_we;
    a.ld_we = ld_we;
    a.N = d_out;
    a.groups = groups;
    a.y = d_y;
    a.y_bf16 = y_dtype == QAMW_BF16;
    a.ld_y = ld_y;
    a.offsets = d_offsets;
    a.experts = experts;
    a.ld_wexpert = ld_wexpert;
    a.ld_weexpert = ld_weexpert;
    a.index = d_index;
    a.x_rows = x_rows;
    return hip_rc(launch_gemm4_grouped(a, (hipStream_t)stream));
}

}  // extern "C"
