/*
 * grouped_ops.h -- C ABI of the products grouped by rows on GB300 (sm_103a):
 * a matrix of its own for each group of rows (experts), with both gradients, and
 * low-rank adapters of many requests beside a shared product.
 *
 * Conventions and element types as in linear_ops.h.  Groups are given by
 * `offsets`, groups + 1 whole numbers in DEVICE memory (int32, or int64 with
 * offsets_type 1): group e has the rows offsets[e] to offsets[e + 1] - 1.  They
 * are read on the device alone.  Each is taken as at least 0, at most `rows` and
 * at least the one before it, so no value of theirs reaches outside the matrices.
 * Rows before offsets[0] and from offsets[groups] on have no group.
 *
 * Types are LINEAR_F16 and LINEAR_BF16; the sums are fp32, results are rounded
 * once.  Widths (N, K) and strides are multiples of 8, pointers 16-byte aligned,
 * row strides at least the rows' width and strides of matrices at least a matrix's
 * extent; up to 1024 groups.  Rows of operands and results may lie between each
 * other's at one stride (slices of one wider matrix).
 */
#ifndef GROUPED_OPS_H
#define GROUPED_OPS_H

#include <stdint.h>

#include "linear_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GROUPED_MAX_GROUPS = 1024 };

/*
 * Options; every zero field means "the default".
 *   tile          rows (of the gradient for the matrices: columns of dD) of a tile:
 *                 16 to 128 (one CTA, by 128 of the other axis), 256 (a CTA pair,
 *                 by 256).  0: chosen from the sizes.
 *   split         1, 2, 4 or 8: a tile's sum is shared by a cluster of so many CTAs,
 *                 one tile each (tiles of 16 to 128); -1: a persistent grid (tiles of
 *                 32 to 256).  0: chosen.  The gradient for the matrices takes tiles
 *                 from 64 on.
 *   max_clusters  cap on the persistent grid (CTAs, or pairs); 0: as many as fit.
 *   debug_flags   test hook: 1 makes every wait run out (see gemm_f16.h).
 *   timeout_ns    limit of every wait inside the kernel; 0: 4 s.
 */
typedef struct grouped_options {
    int32_t tile;
    int32_t split;
    int32_t max_clusters;
    int32_t debug_flags;
    int64_t timeout_ns;
} grouped_options;

/*
 * D[r] = A[r] * B[e]^T for the rows r of group e: A rows x K (`lda` elements
 * apart), B groups matrices of N x K (rows `ldb` apart, matrices `b_stride`), D
 * rows x N (`ldd` apart), of which rows without a group become 0 if `zero_rest`
 * and else are left as they were.  D overlaps no input.  K 0: the groups'
 * rows are 0.
 */
int grouped_gemm_nt(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride, const void *offsets,
                    int32_t offsets_type, void *D, int64_t ldd, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, int32_t zero_rest, void *stream, const grouped_options *opts);

/* Its gradient for A: dA[r] = dD[r] * B[e], dD rows x N, dA rows x K. */
int grouped_gemm_nn(const void *dD, int64_t ldd, const void *B, int64_t ldb, int64_t b_stride, const void *offsets,
                    int32_t offsets_type, void *dA, int64_t lda, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, int32_t zero_rest, void *stream, const grouped_options *opts);

/*
 * Its gradient for B: dB[e] = dD_e^T * A_e over the rows of group e (0 for a group
 * without rows; rows without a group are not read into any sum, whatever they
 * hold).
 */
int grouped_gemm_tn(const void *dD, int64_t ldd, const void *A, int64_t lda, const void *offsets, int32_t offsets_type,
                    void *dB, int64_t ldb, int64_t b_stride, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, void *stream, const grouped_options *opts);

/*
 * A shared product and, beside it, each row's low-rank adapter:
 *
 *     D[r] = x[r] * W^T + scales[a] * (x[r] * down[a]^T) * up[a]^T
 *
 * for the rows r of request e (offsets as above), a = adapters[e] (int32, DEVICE
 * memory); without the second term where a is not in [0, adapter_count) and for rows
 * without a request.  x rows x K, W N x K, down adapter_count matrices of rank x K,
 * up of N x rank, scales fp32 in DEVICE memory (NULL: 1).  scales * (x * down^T), any finite
 * fp32 number, is held as two 16-bit numbers: of LINEAR_BF16 to 2^-16 of itself, of
 * LINEAR_F16 to 2^-22 of its row's largest.  The sum is fp32, D rounded once.  rank is a multiple of 8 up to 128.
 * No row's result depends on another row's adapter.  `workspace`
 * (gemm_lora_workspace_size() bytes, 16-byte aligned, no initialisation, not shared
 * by calls that may overlap on the GPU) holds x * down^T; GEMM_ERR_SCRATCH_LIMIT if it
 * is smaller.  D overlaps no input.  opts: tiles of 16 to 128 take each row's
 * adapter (split 1 to 8), 256 tiles of one request each (split -1).
 */
int gemm_lora_nt(const void *x, int64_t ldx, const void *W, int64_t ldw, const void *down, int64_t ld_down,
                 int64_t down_stride, const void *up, int64_t ld_up, int64_t up_stride, const float *scales,
                 const void *offsets, int32_t offsets_type, const int32_t *adapters, void *D, int64_t ldd, int64_t rows,
                 int64_t requests, int64_t adapter_count, int64_t N, int64_t K, int64_t rank, int32_t type,
                 void *workspace, int64_t workspace_bytes, void *stream, const grouped_options *opts);

/* Bytes of workspace for those sizes, or a negative gemm_status_t. */
int64_t gemm_lora_workspace_size(int64_t rows, int64_t rank);

/*
 * As gemm_f16_last_device_status(), for the calls above: synchronises `stream`,
 * returns and clears the current device's status word.
 */
int grouped_last_device_status(void *stream, uint64_t *info);

#ifdef __cplusplus
}
#endif

#endif /* GROUPED_OPS_H */
