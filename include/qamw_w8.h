/*
 * qamw_w8.h -- 8-bit integer linear layers of libqamw.so, on AMD Instinct MI355X (gfx950).
 *
 * The uniform 8-bit counterpart of the weight codec of qamw.h, for weights and activations alike:
 * rows of a matrix as int8 codes with one fp32 scale a row (an output channel of the weights, a token
 * of the activations), the norm in front of a linear layer with its output in that form, and the
 * product of two matrices in that form.  A linear layer is then
 *     qamw_rmsnorm8 or qamw_quant8 (activations, each call) -> qamw_gemm8 with weights from
 *     qamw_quant8 (once),
 * and, with the channel scales s_j of qamw_act_scale, weights are quantized as w_ij s_j (d_scale of
 * qamw_quant8) and activations as x_j / s_j (1 / s_j folded into d_weight of qamw_rmsnorm8, or as the
 * d_scale of qamw_quant8).  qamw_gemm8 takes any number of activation rows; qamw_qgemm of qamw.h, on
 * the codec's packed weights, at most 16.
 *
 * The conventions of qamw.h hold: caller-owned device pointers, work queued on `stream` of the current
 * device only, no allocation, no state, return codes QAMW_*, faults in the data as bits of *d_status.
 *
 * Codes.  Row i of a code matrix is d int8 values at d_q + i * ld_q.  d_q is 16-byte aligned and ld_q is
 * a multiple of 16, at least d; every row, the last one too, has the bytes up to the next multiple of
 * 16 past d in the buffer: they are written as 0 by qamw_quant8 and qamw_rmsnorm8, and their values do not
 * matter to qamw_dequant8 and qamw_gemm8.  Code q of a row with scale s stands for q s.
 *
 * How a row is quantized.  For a row of fp32 values a_j with largest magnitude top:
 *     s   = fl32(top / 127)                          (row scale)
 *     q_j = rint(fl32(a_j fl32(127 / top)))          (ties to even; -127 .. 127)
 * A row with top < 2^-119 is a zero row: s = 0 and all codes 0.  A row with a value that is not finite
 * sets QAMW_FLAG_NONFINITE, gets s = NaN and all codes 0, so that everything computed from it is NaN.
 */
#ifndef QAMW_W8_H
#define QAMW_W8_H

#include "qamw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row of qamw_quant8 and qamw_rmsnorm8: a row is held in the registers of one workgroup. */
#define QAMW_W8_MAX_COLS 32768

/* Bytes from one row of codes to the next when rows are packed: d rounded up to 16; 0 for d <= 0. */
size_t qamw_q8_stride(int32_t d);

/* Quantize the rows of a matrix (weights, activations, or gated activations).  For every row i:
 *     a_j = x_ij                                       without d_gate
 *         = fl32(x_ij silu(g_ij))                      with d_gate, silu(g) = g / (1 + exp(-g)) in fp32
 *                                                      (to within (|g| + 8) 2^-23 of itself; 0 where
 *                                                      exp(-g) exceeds 2^126)
 *     a_j = fl32(a_j s_j)                              with d_scale
 * then codes and row scale as above.
 *   d_x, x_dtype, ld_x   rows x d values (QAMW_F32 or QAMW_BF16), ld_x >= d; any alignment of rows.
 *   d_gate, ld_gate      NULL, or rows x d gate values of the same type, ld_gate >= d.
 *   d_scale              NULL, or d fp32 channel scales s_j > 0; one that is not sets QAMW_FLAG_BAD_SCALE.
 *   d_q, ld_q            codes; they overlap no input.
 *   d_row_scale          rows fp32.
 * 0 <= rows <= QAMW_MAX_ROWS, 1 <= d <= QAMW_W8_MAX_COLS (QAMW_ERR_UNSUPPORTED above). */
int qamw_quant8(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_gate,
                int64_t ld_gate, const float* d_scale, int8_t* d_q, int64_t ld_q, float* d_row_scale,
                int32_t* d_status, void* stream);

/* The values that codes stand for:
 *     x^_ij = fl32(q_ij s_i), then times fl32(1 / s_j) in fp32 with d_scale (the d_scale of qamw_quant8),
 * rounded to nearest even for QAMW_BF16.  d_out: rows x d, ld_out >= d, any alignment of rows.
 * 0 <= rows <= QAMW_MAX_ROWS, 1 <= d <= QAMW_MAX_ROWS (QAMW_ERR_UNSUPPORTED above). */
int qamw_dequant8(const int8_t* d_q, int32_t rows, int32_t d, int64_t ld_q, const float* d_row_scale,
                  const float* d_scale, void* d_out, qamw_dtype out_dtype, int64_t ld_out, void* stream);

/* Residual addition and root-mean-square norm, with the normalized rows in 8 bits.  For every row i:
 *     h_j = fl32(x_ij + r_ij), or x_ij without d_residual
 *     y_j = h_j w_j / sqrt(sum_j h_j^2 / d + eps)
 * and y as codes and row scale.  The norm is a factor of the whole row, so codes are those of the row
 * a_j = fl32(h_j w_j) (and a zero row is one with all |a_j| < 2^-119), and
 *     s = fl32(top / (127 sqrt(sum_j h_j^2 / d + eps)))
 * with the sum and this quotient in fp64.  h is rounded only where it is stored.
 *   d_x, d_residual   rows x d values of x_dtype (d_residual may be NULL), ld_x, ld_res >= d.
 *   d_weight          d fp32 factors w_j, or NULL for all ones.
 *   eps               finite, >= 0.
 *   d_sum, ld_sum     NULL, or rows x d of x_dtype for h (rounded to nearest even for QAMW_BF16),
 *                     ld_sum >= d; it may be d_x or d_residual itself, with the same ld, and otherwise
 *                     overlaps neither.
 *   d_q .. d_status   as qamw_quant8.
 * Sizes as qamw_quant8. */
int qamw_rmsnorm8(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_residual,
                  int64_t ld_res, const float* d_weight, float eps, void* d_sum, int64_t ld_sum, int8_t* d_q,
                  int64_t ld_q, float* d_row_scale, int32_t* d_status, void* stream);

/* Product of 8-bit matrices with a scale for each token and each output channel:
 *     y[m][n] = fl32(fl32(fl32(c_mn) xs_m) ws_n),   c_mn = sum_k xq[m][k] wq[n][k]
 * with the sum exact in 32 bits (codes may be -128), rounded to nearest even for QAMW_BF16.
 *   d_xq, ld_x, d_xs    M x d_in codes and M fp32 token scales.
 *   d_wq, ld_w, d_wscale   d_out x d_in codes and d_out fp32 channel scales.
 *   d_y, y_dtype, ld_y  M x d_out, ld_y >= d_out; it overlaps no input.
 *   d_ws, ws_bytes      at least qamw_gemm8_workspace(M, d_out, d_in) bytes, 256-byte aligned (may be
 *                       NULL where that is 0); nothing in it has to start at zero.  Calls that may
 *                       overlap (on two streams, in two captured graphs) need one each.
 * 0 <= M, d_out <= QAMW_GEMM8_MAX_ROWS, 1 <= d_in <= QAMW_GEMM8_MAX_COLS (32-bit sums are exact up to
 * there), M * d_out <= QAMW_GEMM8_MAX_OUT, ld_x and ld_w <= QAMW_GEMM8_MAX_LD (QAMW_ERR_UNSUPPORTED above).
 * M = 0 or d_out = 0 is a no-op. */
#define QAMW_GEMM8_MAX_ROWS (1 << 24)
#define QAMW_GEMM8_MAX_COLS 131071
#define QAMW_GEMM8_MAX_LD (1 << 22)
#define QAMW_GEMM8_MAX_OUT (1ll << 38)
size_t qamw_gemm8_workspace(int32_t M, int32_t d_out, int32_t d_in);
int qamw_gemm8(const int8_t* d_xq, int64_t ld_x, const float* d_xs, int32_t M, const int8_t* d_wq, int64_t ld_w,
               const float* d_wscale, int32_t d_out, int32_t d_in, void* d_y, qamw_dtype y_dtype, int64_t ld_y,
               void* d_ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QAMW_W8_H */
