/*
 * fp4mi_ops.h -- operators over the layouts of fp4mi.h for AMD Instinct
 * MI355X (gfx950): matrix products that read MXFP4 rows, FP8 rows and FP8
 * columns, and the RMS norm that produces such rows.
 *
 * Part of libfp4mi.so, under the conventions of fp4mi.h: asynchronous on the
 * given stream, status codes from host-side validation before any launch,
 * caller-owned dense row-major device memory, no state between calls, a call
 * whose output is empty is a no-op that returns FP4_OK.
 *
 * Row formats (FP4_ROWS_*):
 *   MXFP4  codes [rows, cols/2] (two per byte) and UE8M0 bytes [rows, cols/32]
 *          (value 2^(b-127)), as fp4_quantize writes them; cols % 32 == 0.
 *   FP8    E4M3 bytes [rows, cols] and fp32 scales [rows, cols/128], as
 *          mxfp4_row_to_fp8_row writes them; cols % 128 == 0.  The scales are
 *          powers of two in [2^-127, 2^127]; the products read only their
 *          exponent bits.
 *
 * Products accumulate in fp32 and round once to the output type.  A UE8M0 byte
 * of 0xFF or an E4M3 NaN code makes the outputs that read it NaN; FP4_E* is
 * never returned for what a tensor holds.
 */
#ifndef FP4MI_OPS_H
#define FP4MI_OPS_H

#include "fp4mi.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP4_ROWS_MXFP4 0
#define FP4_ROWS_FP8   1

/*
 * mxfp4_matmul -- C[M, N] = diag(r) . A[M, K] . B[N, K]^T.
 *
 *  a, a_fmt      A in row format a_fmt; 16-byte aligned
 *  a_scales      its block scales; 4-byte aligned
 *  a_row_scale   fp32 [M], 4-byte aligned: r, a factor of each row of A (the
 *                row_scale that rmsnorm_quantize writes), or NULL for 1
 *  b, b_scales   B in MXFP4; 16- and 4-byte aligned
 *  M, N          >= 0, below 2^26;  0 < K < 2^21, K % 32 == 0 (MXFP4 A) or
 *                K % 128 == 0 (FP8 A)
 *  out           [M, N] in out_dtype, 16-byte aligned; must not overlap an input
 *
 * The input gradient dX = dY . W of a layer with weights W[N, K] is the same
 * call on W^T quantized along its own rows.
 */
int mxfp4_matmul(const void* a, int a_fmt, const void* a_scales, const float* a_row_scale,
                 const uint8_t* b, const uint8_t* b_scales, int64_t M, int64_t N, int64_t K,
                 void* out, int out_dtype, void* stream);

/*
 * mxfp4_matmul_grouped -- the product per expert over ragged shards: for
 * expert e and tokens t in [off[e], off[e+1])
 *   C[t, :] = r[t] A[t, :] . W[e]^T.
 *
 *  a, a_fmt, a_scales, a_row_scale   as mxfp4_matmul, over all T tokens
 *  w, w_scales    MXFP4 [E, N, K]; 16- and 4-byte aligned
 *  token_offsets  device int64 [E+1]: off[0] = 0, nondecreasing, off[E] = T;
 *                 8-byte aligned (contents are not validated on the host;
 *                 malformed offsets are clamped on the device: rows outside
 *                 every shard are then not written, the others are
 *                 unspecified, and every access stays inside the buffers)
 *  num_experts    1 <= E < 2^23 (FP4_EINVAL below 1, FP4_ESHAPE from 2^23);
 *                 0 <= T < 2^26;  N, K as above
 *  out            [T, N] in out_dtype, 16-byte aligned; must not overlap an input
 */
int mxfp4_matmul_grouped(const void* a, int a_fmt, const void* a_scales, const float* a_row_scale,
                         const uint8_t* w, const uint8_t* w_scales, const int64_t* token_offsets,
                         int32_t num_experts, int64_t total_tokens, int64_t N, int64_t K,
                         void* out, int out_dtype, void* stream);

/*
 * fp8_matmul_tokblk -- the weight gradient per expert, contracting over the
 * expert's tokens:
 *   out[e] = A_e . B_e^T,  A_e [M, n_e], B_e [N, n_e],
 * both operands in the layout that mxfp4_row_to_fp8_col_tokblk writes (E4M3
 * columns dense per expert, power-of-two fp32 scales per channel and block of
 * 128 tokens).  For a layer Y = X . W^T with W[e] [M, N], A holds dY's columns
 * and B holds X's.  An expert without tokens gets zeros.
 * No factor per token is applied: where Y took one (the products' a_row_scale
 * r, so Y = diag(r) . X . W^T), dY's rows are multiplied by it before they are
 * quantized.  dY's columns without it give another gradient, with no error.
 *
 *  a, b           bytes [T * M], [T * N], 4-byte aligned
 *  a_scales, b_scales  fp32 [M (ceil(T/128) + E)], [N (ceil(T/128) + E)],
 *                 4-byte aligned
 *  token_offsets, num_experts  as mxfp4_matmul_grouped;  0 <= T < 2^24
 *  M, N           >= 0, below 2^21, % 128 == 0
 *  out            [E, M, N] in out_dtype, 16-byte aligned; must not overlap an input
 */
int fp8_matmul_tokblk(const uint8_t* a, const float* a_scales, const uint8_t* b,
                      const float* b_scales, const int64_t* token_offsets, int32_t num_experts,
                      int64_t total_tokens, int64_t M, int64_t N, void* out, int out_dtype,
                      void* stream);

/*
 * rmsnorm_quantize -- residual addition, RMS norm and quantized rows.
 *
 * Per row, with x and residual widened to fp32:
 *   h = x + residual, rounded to x's dtype (x itself without a residual);
 *   row_scale = 1 / sqrt(mean(h^2) + eps);
 *   z = fl32(h * weight), quantized to rows of format fmt (RTN).
 * The normalized row is row_scale * (codes * block scale): the factor that
 * depends on the whole row is kept apart as one fp32, for the products'
 * a_row_scale, so codes and block scales are those of z exactly.  The rows
 * alone are not normalized: whatever reads them takes row_scale as a factor,
 * the weight gradient by way of dY (fp8_matmul_tokblk; it reads columns, which
 * are made from MXFP4 rows).
 *   MXFP4: as fp4_quantize.  FP8: the scale of 128 values is the least power
 *   of two 2^k, -126 <= k <= 127, with max|z| <= 448 * 2^k (2^-127 for a block
 *   of zeros), and the code is E4M3(z / 2^k), to nearest even, saturating.
 * Where h or z is infinite or NaN the row's outputs are unspecified.  The sum
 * of squares is taken in fp32: row_scale is 0 where it passes fp32's range (some
 * |h| from 2^64), and squares below 2^-149 count as 0.
 *
 *  x, residual   [rows, cols] in dtype, 16-byte aligned; residual may be NULL
 *  weight        [cols] in weight_dtype, 16-byte aligned
 *  rows, cols    rows >= 0; 0 < cols < 2^21, cols % 32 == 0 (MXFP4) or % 128 == 0
 *  eps           >= 0, finite
 *  fmt           FP4_ROWS_MXFP4 or FP4_ROWS_FP8
 *  q, scales     out, in the layout of fmt; q 16-byte, scales 4-byte aligned
 *  row_scale     out fp32 [rows], 4-byte aligned
 *  h             out [rows, cols] in dtype, 16-byte aligned, or NULL; may be x
 *                or residual itself, no other output may overlap an input
 */
int rmsnorm_quantize(const void* x, const void* residual, int dtype, const void* weight,
                     int weight_dtype, int64_t rows, int64_t cols, float eps, int fmt, void* q,
                     void* scales, float* row_scale, void* h, void* stream);

/*
 * rmsnorm_backward -- gradient of y = row_scale * h * weight (rounding to the
 * row format passed straight through), with r = row_scale:
 *   g = dy * weight;
 *   dx = r (g - h r^2 mean(g h)) [+ dh];   dweight = sum over rows of dy h r.
 * dx is the gradient of x and of the residual alike.
 *
 *  dy, h         [rows, cols] in dtype, 16-byte aligned
 *  dh            the gradient that reaches h past the norm, same layout, or NULL
 *  weight        [cols] in weight_dtype, 16-byte aligned
 *  row_scale     fp32 [rows], as rmsnorm_quantize wrote it
 *  rows, cols    rows >= 0; 0 < cols < 2^21, cols % 32 == 0
 *  dx            out [rows, cols] in dtype, 16-byte aligned; may be dy or dh itself
 *  dweight       out fp32 [cols], 16-byte aligned (zeros when rows == 0)
 *  workspace     scratch of rmsnorm_backward_workspace(rows, cols) bytes or more
 *                (workspace_bytes; FP4_ESHAPE if fewer), 16-byte aligned; holds
 *                partial sums that are added in a fixed order, so results do
 *                not vary between calls
 */
int rmsnorm_backward(const void* dy, const void* h, const void* dh, int dtype, const void* weight,
                     int weight_dtype, const float* row_scale, int64_t rows, int64_t cols, void* dx,
                     float* dweight, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of rmsnorm_backward's workspace (0 for sizes it refuses). */
int64_t rmsnorm_backward_workspace(int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif

#endif /* FP4MI_OPS_H */
