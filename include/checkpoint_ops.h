/*
 * checkpoint_ops.h -- C ABI of layer norm that keeps 8 bits an element for its
 * backward pass, on GB300 (sm_103a).
 *
 * Conventions and element types as in linear_ops.h.  In place of its input x
 * (and of its result, for the product behind it) the norm keeps its normalised rows
 *
 *     h[j] = (x[j] - mean) * rstd
 *
 * as microscaled 8-bit floats, from which both the result and the gradient follow:
 *   codes   [rows][cols] bytes, E4M3
 *   scales  [rows][ceil(cols / 32)] bytes, E8M0 (2^(code - 127)), one for each 32
 *           elements of a row: 2^(floor(log2(amax)) - 8), amax the block's largest
 *           magnitude, the exponent at least -127 (the conversion of the OCP
 *           Microscaling Formats specification v1.0)
 * The value of an element is E4M3(code) * scale; an element is h / scale rounded
 * to E4M3 (nearest, ties to the even code, magnitudes past 448 to 448).  A block that
 * holds an infinity or NaN has the scale code 255 and stands for NaN.
 */
#ifndef CHECKPOINT_OPS_H
#define CHECKPOINT_OPS_H

#include <stdint.h>

#include "linear_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * layer_norm_forward() that keeps its normalised rows: y, codes, scales and rstd
 * (fp32, `rows`) are written; y may be NULL.  Arguments as there.  Outputs overlap
 * neither inputs nor each other.
 */
int norm_checkpoint_forward(const void *x, int64_t x_stride, const void *weight, const void *bias, void *y,
                            int64_t y_stride, void *codes, void *scales, float *rstd, int64_t rows, int64_t cols,
                            float eps, int32_t type, int32_t weight_type, void *stream);

/*
 * The norm's result from what it kept: y[j] = h[j] * weight[j] + bias[j] for the
 * values h of the codes, rounded once to `type` (weight_type is `type` or LINEAR_F32;
 * weight and bias may be NULL: 1 and 0).  y overlaps no input.
 */
int norm_checkpoint_restore(const void *codes, const void *scales, const void *weight, const void *bias, void *y,
                            int64_t y_stride, int64_t rows, int64_t cols, int32_t type, int32_t weight_type,
                            void *stream);

/*
 * The gradient of the norm from what it kept, as layer_norm_backward() with the
 * values of the codes for h.  `workspace`: layer_norm_backward_workspace_size() bytes.
 */
int norm_checkpoint_backward(const void *dy, int64_t dy_stride, const void *codes, const void *scales, const void *weight,
                             const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias, int64_t rows,
                             int64_t cols, int32_t type, int32_t weight_type, void *workspace, int64_t workspace_bytes,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CHECKPOINT_OPS_H */
