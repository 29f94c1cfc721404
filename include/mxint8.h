/*
 * mxint8.h -- C ABI of activation checkpoints in 8 bits: what training keeps of
 * an activation for its backward pass, in half the bytes of bf16.
 *
 * The format is MXINT8 of the OCP Microscaling Formats specification v1.0.  A
 * matrix [rows][cols] is cut into blocks of 32 consecutive elements of a row; a
 * block has one scale 2^e and each element is an integer of -127 .. 127:
 *
 *   e = max(floor(log2(max |x|)), -127),   q = clamp(rne(x * 2^-e * 64), -127, 127)
 *
 * and stands for q * 2^(e - 6).  rne rounds to nearest, ties to even; the clamp
 * meets what rounds to 128, so |x - value| <= 2^(e - 6).  A block that holds a NaN or
 * an infinity reads as NaN throughout; a block of zeros as zeros.  Seven bits and a
 * power of two fit a bf16 number, so every value is exact in bf16 and in fp32.
 *
 * Memory, for rows x cols with B = ceil(cols/32) blocks to a row:
 *   data    [rows][32*B] int8, zero past cols (the readers need that);
 *   scales  [rows][B] bytes, e + 127; 255 = NaN.
 *
 * The conventions are conv2d.h's (status codes, caller-owned device memory, work
 * enqueued on `stream`, nothing allocated).
 */
#ifndef SPLIT_GEMM_GB300_MXINT8_H
#define SPLIT_GEMM_GB300_MXINT8_H

#include "layer_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of data and of scales for a matrix of rows x cols; 0 where either is below 1 or past 2^31 - 32. */
size_t mxint8_data_bytes(int64_t rows, int64_t cols);
size_t mxint8_scale_bytes(int64_t rows, int64_t cols);

/* Quantises x [rows][cols] (x_dtype: conv2d_out_dtype; x_stride elements from one row to the next; aligned to its
 * element type).  data is 16-byte aligned. */
int mxint8_quantize(int64_t rows, int64_t cols, const void* x_dev, int32_t x_dtype, int64_t x_stride, void* data_dev,
                    void* scales_dev, conv2d_stream_t stream);

/* y [rows][cols], dense, of y_dtype, aligned to its element type: the values that data (16-byte aligned) and scales stand for. */
int mxint8_dequantize(int64_t rows, int64_t cols, const void* data_dev, const void* scales_dev, void* y_dev,
                      int32_t y_dtype, conv2d_stream_t stream);

/* layer_norm_bwd with x as a checkpoint: data (16-byte aligned) and scales in the place of x_dev.  params: rows, cols, y_stride and
 * y_dtype (of dy) are used; dx is dense [rows][cols] of dy's type, may be dy itself where that is dense, and overlaps no other operand. */
size_t mxint8_layer_norm_bwd_workspace_bytes(const layer_norm_params* params);

int mxint8_layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* data_dev, const void* scales_dev,
                          const float* mean_dev, const float* rstd_dev, const float* weight_dev, void* dx_dev,
                          float* dweight_dev, float* dbias_dev, void* workspace_dev, size_t workspace_bytes,
                          conv2d_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLIT_GEMM_GB300_MXINT8_H */
