/*
 * layer_norm.h -- C ABI of layer normalisation over the channels of NHWC
 * activations (or the features of tokens): forward, backward, and forward with
 * a 4-bit microscaled output.
 *
 *   mean[r] = sum_c x[r][c] / C
 *   rstd[r] = 1 / sqrt(sum_c (x[r][c] - mean[r])^2 / C + eps)
 *   y[r][c] = (x[r][c] - mean[r]) * rstd[r] * weight[c] + bias[c]
 *
 * and for an output gradient dy, with xh = (x - mean) * rstd and g = dy * weight:
 *
 *   dx[r][c]   = rstd[r] * (g[r][c] - sum_c g[r][c] / C - xh[r][c] * sum_c (g * xh)[r][c] / C)
 *   dweight[c] = sum_r dy[r][c] * xh[r][c]
 *   dbias[c]   = sum_r dy[r][c]
 *
 * All sums and statistics are fp32; the deviations are taken from the row's own
 * mean (no difference of large squares), and a value is rounded once, where it
 * is stored.  The conventions are conv2d.h's (status codes, caller-owned device
 * memory, work enqueued on `stream`, nothing allocated), except that a pointer
 * need only be aligned to its own element type.  Results do not depend on the
 * order in which blocks run: two calls on the same inputs give the same bits.
 */
#ifndef SPLIT_GEMM_GB300_LAYER_NORM_H
#define SPLIT_GEMM_GB300_LAYER_NORM_H

#include "conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t rows, cols;          /* 0 <= rows < 2^31, 1 <= cols <= 2^30 */
    int64_t x_stride, y_stride;  /* elements from one row to the next, >= cols (y_stride: of y, or of dy) */
    int32_t x_dtype, y_dtype;    /* conv2d_out_dtype of x (and dx), and of y (or dy) */
    float eps;                   /* >= 0 */
} layer_norm_params;

/* y, and mean and rstd [rows] fp32 for the backward pass.  weight_dev, bias_dev:
 * [cols] fp32 or NULL (1 and 0); mean_dev, rstd_dev may be NULL.  y may be x
 * itself when type and stride are the same. */
int layer_norm_fwd(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                   const float* bias_dev, void* y_dev, float* mean_dev, float* rstd_dev, conv2d_stream_t stream);

/* dx [rows][cols], dense, of x's type, overlapping no operand; dweight_dev, dbias_dev [cols] fp32, each
 * may be NULL (not computed); both are zero for no rows.  The sums over the
 * rows are joined in a fixed order.  workspace_dev: at least
 * layer_norm_bwd_workspace_bytes() bytes of any content, 16-byte aligned (may be
 * NULL when that is 0 or neither dweight nor dbias is wanted). */
size_t layer_norm_bwd_workspace_bytes(const layer_norm_params* params);

int layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* x_dev, const float* mean_dev,
                   const float* rstd_dev, const float* weight_dev, void* dx_dev, float* dweight_dev,
                   float* dbias_dev, void* workspace_dev, size_t workspace_bytes, conv2d_stream_t stream);

/* The forward pass with its fp32 result quantised at once (mxfp4.h: data
 * [rows][16*ceil(cols/32)], scales mxfp4_scale_bytes(rows, cols) bytes).
 * y_dtype and y_stride are not used. */
int layer_norm_mxfp4(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                     const float* bias_dev, void* data_dev, void* scales_dev, float* mean_dev, float* rstd_dev,
                     conv2d_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLIT_GEMM_GB300_LAYER_NORM_H */
