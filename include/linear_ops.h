/*
 * linear_ops.h -- C ABI of the operators around a linear layer's product on
 * GB300 (sm_103a): layer norm and its gradient, quantisation to microscaled
 * 4-bit floats, and the product of two such matrices.
 *
 * Conventions (those of gemm_f16.h): pointers are DEVICE pointers owned by the
 * caller; the library keeps none and allocates nothing.  `stream` is a
 * cudaStream_t as void* (NULL = the legacy default stream).  Calls are
 * asynchronous: they validate, enqueue and return.  Errors are the negative
 * gemm_status_t values; an argument error is reported before anything is
 * enqueued.  Row strides are in elements; rows may lie anywhere (a stride of
 * 0, one row read again and again, is allowed for inputs).  Element types:
 */
#ifndef LINEAR_OPS_H
#define LINEAR_OPS_H

#include <stdint.h>

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum linear_dtype { LINEAR_F16 = 0, LINEAR_BF16 = 1, LINEAR_F32 = 2 } linear_dtype_t;

/*
 * Layer norm of `rows` rows of `cols` elements:
 *
 *     mean = sum_j x[j] / cols        rstd = 1 / sqrt(sum_j (x[j] - mean)^2 / cols + eps)
 *     y[j] = (x[j] - mean) * rstd * weight[j] + bias[j]
 *
 * x and y have type `type`; weight and bias (either may be NULL: 1 and 0) have
 * type `weight_type`, which is `type` or LINEAR_F32.  mean and rstd (fp32,
 * `rows` each) may both be NULL.  Sums are fp32, the variance from the centred
 * values; y is rounded once.  cols >= 1, rows >= 0.  y, mean and rstd must not
 * overlap x, weight, bias or each other, nor y its own rows (y_stride >= cols).
 * eps >= 0 and finite.
 * Any alignment of whole elements is accepted; 16-byte aligned rows are faster.
 */
int layer_norm_forward(const void *x, int64_t x_stride, const void *weight, const void *bias, void *y, int64_t y_stride,
                       float *mean, float *rstd, int64_t rows, int64_t cols, float eps, int32_t type,
                       int32_t weight_type, void *stream);

/*
 * Gradient of layer_norm_forward() from what it left (x, mean, rstd):
 *
 *     h = (x - mean) * rstd     g = dy * weight
 *     dx = rstd * (g - sum_j(g) / cols - h * sum_j(g * h) / cols)
 *     dweight[j] = sum_rows dy * h        dbias[j] = sum_rows dy
 *
 * dx has type `type`; weight (NULL: 1), dweight and dbias have `weight_type`;
 * dweight and dbias may both be NULL (not one of them).  Sums over rows are
 * fp32 in a fixed order: the same inputs give the same bits.  `workspace` holds the partial sums
 * (layer_norm_backward_workspace_size() bytes, 16-byte aligned, no
 * initialisation, not shared by calls that may overlap on the GPU);
 * GEMM_ERR_SCRATCH_LIMIT if it is smaller.  The outputs must not overlap the
 * inputs or the workspace.
 */
int layer_norm_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const void *weight,
                        const float *mean, const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                        int64_t rows, int64_t cols, int32_t type, int32_t weight_type, void *workspace,
                        int64_t workspace_bytes, void *stream);

/* Bytes of workspace for those sizes on any device, or a negative gemm_status_t. */
int64_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols);

/*
 * A microscaled 4-bit matrix of rows x cols:
 *   data    [rows][ceil(cols / 32) * 16] bytes: two E2M1 codes a byte, the even
 *           column in the low nibble; columns from `cols` on hold code 0
 *   scales  [ceil(rows / 128)][ceil(blocks / 4)][32][4][4] bytes, blocks =
 *           ceil(cols / 32) * 32 / block: the scale code of row 128 i + 32 g + l
 *           and block 4 j + k is at [i][j][l][g][k]; 0 where there is none.  It
 *           is the order in which the tensor cores take them.
 * The value of an element is E2M1(code) * scale.  Formats:
 *   FP4_MX  blocks of 32 elements of a row, E8M0 scales (2^(code - 127), 255 NaN)
 *   FP4_NV  blocks of 16, E4M3 scales times 2^exponent, one exponent in
 *           [-100, 100] for the whole matrix (0 for FP4_MX)
 */
typedef enum fp4_format { FP4_MX = 0, FP4_NV = 1 } fp4_format_t;

/* Bytes of data and scales of such a matrix; negative gemm_status_t on bad arguments
 * (GEMM_ERR_UNSUPPORTED_SHAPE for more than 2^31 - 1024 rows or 65535 * 4096 columns). */
int64_t fp4_data_bytes(int64_t rows, int64_t cols);
int64_t fp4_scale_bytes(int64_t rows, int64_t cols, int32_t format);

/*
 * Quantise x (rows x cols, `type`).  With amax the block's largest magnitude:
 *   FP4_MX: scale = 2^(floor(log2(amax)) - 2), the exponent kept in [-127, 127]
 *           (the conversion of the OCP Microscaling Formats specification v1.0)
 *   FP4_NV: scale = e * 2^exponent, e = amax / 6 / 2^exponent rounded to E4M3
 *           (nearest, ties to even) within [2^-9, 448]
 * and each element is x / scale rounded to E2M1 (nearest, ties to the even
 * code, magnitudes past 6 to 6).  A block that holds an infinity or NaN gets a
 * NaN scale and codes 0.  Every byte of data and scales is written.
 */
int fp4_quantize(const void *x, int64_t x_stride, int64_t rows, int64_t cols, int32_t type, int32_t format,
                 int32_t exponent, void *data, void *scales, void *stream);

/* The values a quantised matrix stands for, rounded once to `type`. */
int fp4_dequantize(const void *data, const void *scales, int64_t rows, int64_t cols, int32_t format, int32_t exponent,
                   void *out, int64_t out_stride, int32_t type, void *stream);

/*
 * Options of gemm_fp4_nt(); every zero field means "the default".
 *   tile          0: chosen from the shape.  16, 32, 64, 128: one CTA per tile
 *                 of 128 rows of one operand by that many rows of the other.
 *                 256: CTA pairs with 256 x 256 tiles.
 *   cluster_k     single-CTA tiles: K split over a cluster of 1, 2, 4 or 8 CTAs;
 *                 0: chosen.
 *   swap          single-CTA tiles: 1: the 128 rows are A's; 2: they are B's
 *                 (few rows of A, as for single tokens); 0: chosen.  Tiles
 *                 of 16, 32 and 64 are for at most that many rows of the other
 *                 operand.
 *   max_clusters  cap on the persistent grid of CTA pairs; 0: as many as fit.
 *   debug_flags   test hook: 1 makes every wait run out (see gemm_f16.h).
 *   timeout_ns    limit of every wait inside the kernel; 0: 4 s.
 *   exponent      FP4_NV: the result's power of two beside alpha, in [-1000,
 *                 1000] (0 for FP4_MX).
 */
typedef struct gemm_fp4_options {
    int32_t tile;
    int32_t cluster_k;
    int32_t swap;
    int32_t max_clusters;
    int32_t debug_flags;
    int64_t timeout_ns;
    int32_t exponent;
} gemm_fp4_options;

/*
 * D = alpha * 2^exponent * A * B^T for quantised A (M x K) and B (N x K) of one
 * format, K their number of columns; D (M x N, row-major, `d_type`) is rounded
 * once from the fp32 sum of codes times scales, times alpha * 2^exponent.  The
 * exponents of FP4_NV matrices, which the kernel does not see, belong there: into
 * the option (exponent of A + exponent of B), as their sum may leave fp32's range,
 * or into alpha where it does not.  A, B and their scales are
 * 16-byte aligned; D is aligned to its elements (16-byte aligned rows are
 * faster) and overlaps none of them.  M or N 0: nothing is launched; K 0:
 * D = 0.  M, N <= 2^31 - 1024, K as the columns of a quantised matrix.
 */
int gemm_fp4_nt(const void *A, const void *A_scales, const void *B, const void *B_scales, void *D, int64_t M, int64_t N,
                int64_t K, int32_t format, int32_t d_type, float alpha, void *stream, const gemm_fp4_options *opts);

/* What gemm_fp4_nt() would launch on a device of `sm_count` SMs; pure host logic. */
typedef struct gemm_fp4_launch_info {
    int32_t tile, cluster_k, swap;
    int64_t ctas;
} gemm_fp4_launch_info;
int gemm_fp4_nt_describe(int64_t M, int64_t N, int64_t K, int32_t format, const gemm_fp4_options *opts,
                         int32_t sm_count, gemm_fp4_launch_info *out);

/*
 * As gemm_f16_last_device_status(), for gemm_fp4_nt(): synchronises `stream`,
 * returns and clears the current device's status word (GEMM_OK or
 * GEMM_ERR_DEVICE_TIMEOUT; `info`, if not NULL, says where).
 */
int gemm_fp4_last_device_status(void *stream, uint64_t *info);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_OPS_H */
