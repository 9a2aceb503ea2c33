/*
 * qamw_mx4.h -- microscaled 4-bit linear layers of libqamw.so, on AMD Instinct MI355X (gfx950).
 *
 * The 4-bit floating-point counterpart of the 8-bit layers of qamw_w8.h: rows of a matrix as 4-bit codes with
 * a power of two for every 32 columns, the norm in front of a linear layer with its output in that form, the
 * product of two matrices in that form, and the same product for rows in groups with weights of their own (the
 * experts of a mixture).  A linear layer is
 *     qamw_rmsnorm4 or qamw_quant4 (activations, each call) -> qamw_gemm4 or qamw_gemm4_grouped with weights
 *     from qamw_quant4 (once),
 * with channel scales s_j (qamw_act_scale) as for the 8-bit layers: weights are quantized as w_ij s_j (d_scale of
 * qamw_quant4) and activations as x_j / s_j (1 / s_j folded into d_weight of qamw_rmsnorm4, or as d_scale).
 *
 * The conventions of qamw.h hold: caller-owned device pointers, work queued on `stream` of the current
 * device only, no allocation, no state, return codes QAMW_*, faults in the data as bits of *d_status.
 *
 * The form.  A matrix of `rows` rows and d columns has kt = ceil(d / 256) groups of 256 columns.
 *   Codes: row i is qamw_mx4_stride(d) = 128 kt bytes at d_q + i * ld_q, two columns a byte, column 2b in bits 0-3
 *   of byte b and column 2b+1 in bits 4-7.  Code c stands for (-1)^(c / 8) times entry c % 8 of
 *   0, 0.5, 1, 1.5, 2, 3, 4, 6.  d_q is 16-byte aligned, ld_q a multiple of 16 and at least the stride.
 *   Scales: block b of a row (columns 32 b .. 32 b + 31) has the byte at d_e + (b / 8) * ld_e + i * 8 + b % 8, and
 *   every code of the block is times 2^(byte - 127); byte 255 makes the block NaN.  d_e is 8-byte aligned, ld_e a
 *   multiple of 8 and at least 8 rows.  (Groups stand outermost: the rows that a product reads together have
 *   their scales together.)  Bytes of other origin that stand by rows, one for every 32 columns, are brought into this
 *   order by zeros up to 8 kt bytes a row and exchanging rows and groups of 8 bytes; their codes need zeros up to 128 kt.
 * qamw_quant4 and qamw_rmsnorm4 write whole groups: codes past d are 0, scale bytes of blocks past d are 0.
 * The products take whole groups: their sums run over all 256 kt columns.
 *
 * How a block is quantized.  For 32 fp32 values a_j (0 past d) with largest magnitude top:
 *     E the least integer with top <= 7 2^E,  byte = E + 127,
 *     code_j = the nearest of the values above to |a_j| 2^-E, ties to the even code, above 6 to 6, bit 3 the sign
 *              of a_j
 * (up to 7, a value is no further from 6 than a value below 6 may be from its code).  A block with
 * top < 2^-119 has byte 0 and codes 0.  A block with a value that is not finite sets QAMW_FLAG_NONFINITE and
 * has byte 255 and codes 0, so that everything computed from it is NaN.
 */
#ifndef QAMW_MX4_H
#define QAMW_MX4_H

#include "qamw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest rows: of qamw_rmsnorm4, which holds a row in the registers of one workgroup, and of everything else. */
#define QAMW_MX4_MAX_NORM_COLS 32768
#define QAMW_MX4_MAX_COLS (1 << 23)

/* Bytes of a row of codes: 128 for every 256 columns or part of them; 0 for d <= 0. */
size_t qamw_mx4_stride(int32_t d);

/* Groups of 256 columns: ceil(d / 256); 0 for d <= 0. */
int32_t qamw_mx4_groups(int32_t d);

/* Quantize the rows of a matrix (weights, activations, or gated activations).  For every row i:
 *     a_j = x_ij                                       without d_gate
 *         = fl32(x_ij g_ij / (1 + exp(-g_ij)))         with d_gate: in fp64 (to within 2^-38 of itself), rounded
 *                                                      to fp32 once
 *     a_j = fl32(a_j s_j)                              with d_scale
 * then blocks as above.
 *   d_x, x_dtype, ld_x   rows x d values (QAMW_F32 or QAMW_BF16), ld_x >= d; any alignment of rows.
 *   d_gate, ld_gate      NULL, or rows x d gate values of the same type, ld_gate >= d.
 *   d_scale              NULL, or d fp32 channel scales s_j > 0; one that is not sets QAMW_FLAG_BAD_SCALE.
 *   d_q, ld_q, d_e, ld_e codes and scales; they overlap no input.
 * 0 <= rows <= QAMW_MAX_ROWS, 1 <= d <= QAMW_MX4_MAX_COLS (QAMW_ERR_UNSUPPORTED above). */
int qamw_quant4(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_gate,
                int64_t ld_gate, const float* d_scale, uint8_t* d_q, int64_t ld_q, uint8_t* d_e, int64_t ld_e,
                int32_t* d_status, void* stream);

/* The values that codes stand for:
 *     x^_ij = value(code_ij) 2^(byte - 127) in fp32, then times fl32(1 / s_j) in fp32 with d_scale (the d_scale of
 *     qamw_quant4),
 * rounded to nearest even for QAMW_BF16.  (A code of 4 or 6 with byte 253 or 254, which only values of
 * 3.5 2^126 and more get, reads back as infinity.)  d_out: rows x d, ld_out >= d, any alignment of rows.  Sizes as
 * qamw_quant4. */
int qamw_dequant4(const uint8_t* d_q, int32_t rows, int32_t d, int64_t ld_q, const uint8_t* d_e, int64_t ld_e,
                  const float* d_scale, void* d_out, qamw_dtype out_dtype, int64_t ld_out, void* stream);

/* Residual addition and root-mean-square norm, with the normalized rows in 4 bits.  For every row i:
 *     h_j = fl32(x_ij + r_ij), or x_ij without d_residual
 *     f   = fl32(1 / sqrt(sum_j h_j^2 / d + eps)), in fp64 but for that rounding
 *     a_j = fl32(fl32(h_j w_j) f)
 * then blocks as above.  h is rounded only where it is stored.  The sum's order goes by rows and d: where 1 / sqrt(..) is
 * within about d 2^-53 of the middle of two fp32 numbers, f may be the one in one call and the other in a call of more
 * rows, and codes that lie next to a border may differ.  Calls of the same sizes give the same codes.
 *   d_x, d_residual   rows x d values of x_dtype (d_residual may be NULL), ld_x, ld_res >= d.
 *   d_weight          d fp32 factors w_j, or NULL for all ones.
 *   eps               finite, >= 0.  (A row of zeros with eps = 0 has f infinite and a_j NaN: it is flagged.)
 *   d_sum, ld_sum     NULL, or rows x d of x_dtype for h (rounded to nearest even for QAMW_BF16),
 *                     ld_sum >= d; it may be d_x or d_residual itself, with the same ld, and otherwise
 *                     overlaps neither.
 *   d_q .. d_status   as qamw_quant4.
 * 0 <= rows <= QAMW_MAX_ROWS, 1 <= d <= QAMW_MX4_MAX_NORM_COLS (QAMW_ERR_UNSUPPORTED above). */
int qamw_rmsnorm4(const void* d_x, qamw_dtype x_dtype, int32_t rows, int32_t d, int64_t ld_x, const void* d_residual,
                  int64_t ld_res, const float* d_weight, float eps, void* d_sum, int64_t ld_sum, uint8_t* d_q,
                  int64_t ld_q, uint8_t* d_e, int64_t ld_e, int32_t* d_status, void* stream);

/* Product of two matrices in 4 bits:
 *     y[m][n] = sum_k x^[m][k] w^[n][k]     over 256 `groups` columns
 * on the matrix cores, which add the products of 64 columns (exact each) at a time to an fp32 sum, within 2^-23 of the
 * largest of the sum's and the products' summed magnitudes; the parts of k that a size is split into are added in a
 * fixed order, so results do not depend on timing.  y is rounded to nearest even for QAMW_BF16.  The two scale bytes of a
 * product count together, so that neither alone leaves the range of fp32; the sums are fp32 numbers: below the normal ones
 * they are multiples of 2^-149, and one past the range is infinite, or NaN behind another.  A block with scale byte
 * 255 makes its row of x, or its column of y, NaN.
 *   d_xq, ld_x, d_xe, ld_xe    M rows of codes and their scales.
 *   d_wq, ld_w, d_we, ld_we    d_out rows of codes and their scales.
 *   d_y, y_dtype, ld_y  M x d_out, ld_y >= d_out; it overlaps no input.
 *   d_ws, ws_bytes      at least qamw_gemm4_workspace(M, d_out, groups) bytes, 256-byte aligned (may be
 *                       NULL where that is 0); nothing in it has to start at zero.  Calls that may
 *                       overlap (on two streams, in two captured graphs) need one each.
 * 0 <= M, d_out <= QAMW_GEMM4_MAX_ROWS, 1 <= groups <= QAMW_MX4_MAX_COLS / 256, M * d_out <= QAMW_GEMM4_MAX_OUT,
 * ld_x and ld_w <= QAMW_GEMM4_MAX_LD (QAMW_ERR_UNSUPPORTED above).  M = 0 or d_out = 0 is a no-op. */
#define QAMW_GEMM4_MAX_ROWS (1 << 24)
#define QAMW_GEMM4_MAX_LD (1 << 22)
#define QAMW_GEMM4_MAX_OUT (1ll << 38)
size_t qamw_gemm4_workspace(int32_t M, int32_t d_out, int32_t groups);
int qamw_gemm4(const uint8_t* d_xq, int64_t ld_x, const uint8_t* d_xe, int64_t ld_xe, int32_t M, const uint8_t* d_wq,
               int64_t ld_w, const uint8_t* d_we, int64_t ld_we, int32_t d_out, int32_t groups, void* d_y,
               qamw_dtype y_dtype, int64_t ld_y, void* d_ws, size_t ws_bytes, void* stream);

/* The product for rows in groups (a mixture of experts): row i of y, for offsets[e] <= i < offsets[e + 1], is
 *     y[i][n] = sum_k x^[r_i][k] w^_e[n][k],    r_i = index[i], or i without d_index,
 * with the weights w^_e of expert e.  Groups may have any sizes, none too; what they are is read on the device, so
 * that a router's result needs no copy to the host.
 *   d_xq, ld_x, d_xe, ld_xe, x_rows   x_rows rows of codes and their scales.
 *   d_index      NULL (then x_rows >= rows), or `rows` row numbers of x, in any order and any number of times; one
 *                outside 0 .. x_rows - 1 stands for a row of zeros.
 *   rows         rows of y.  Those that no group has (before offsets[0], from offsets[experts] on) are left as they
 *                were.
 *   d_wq, ld_w, ld_wexpert    row n of expert e is at d_wq + e * ld_wexpert + n * ld_w: ld_wexpert a multiple of 16,
 *                at least 0.
 *   d_we, ld_we, ld_weexpert  its scales at d_we + group * ld_we + e * ld_weexpert + n * 8: ld_weexpert a multiple of
 *                8, at least 0.
 *   d_offsets    experts + 1 int32, non-decreasing, from 0 to rows.  Values outside that range count as its nearest
 *                end, and a group that ends before it begins is empty; where groups overlap all the same, the rows
 *                that more than one has, and any behind the first overlap, are unspecified.
 *   d_y, y_dtype, ld_y  rows x d_out, ld_y >= d_out; it overlaps no input.
 * Limits of qamw_gemm4 for rows, x_rows, d_out, groups and leading dimensions; 1 <= experts <=
 * QAMW_GEMM4_MAX_EXPERTS, experts * d_out <= QAMW_GEMM4_MAX_EXPERT_ROWS, and with d_index x_rows * ld_x <=
 * QAMW_GEMM4_MAX_INDEXED bytes (QAMW_ERR_UNSUPPORTED above).  rows = 0 or d_out = 0 is a no-op. */
#define QAMW_GEMM4_MAX_EXPERTS 1024
#define QAMW_GEMM4_MAX_EXPERT_ROWS (1 << 30)
#define QAMW_GEMM4_MAX_INDEXED (1ll << 31)
int qamw_gemm4_grouped(const uint8_t* d_xq, int64_t ld_x, const uint8_t* d_xe, int64_t ld_xe, int32_t x_rows,
                       const int32_t* d_index, int32_t rows, const uint8_t* d_wq, int64_t ld_w, int64_t ld_wexpert,
                       const uint8_t* d_we, int64_t ld_we, int64_t ld_weexpert, const int32_t* d_offsets,
                       int32_t experts, int32_t d_out, int32_t groups, void* d_y, qamw_dtype y_dtype, int64_t ld_y,
                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QAMW_MX4_H */
