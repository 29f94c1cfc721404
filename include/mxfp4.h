/*
 * mxfp4.h -- C ABI of microscaled 4-bit matrices: quantisation, the way back,
 * and the matrix product (a pointwise convolution of NHWC rows).
 *
 * The format is MXFP4 of the OCP Microscaling Formats specification v1.0.  A
 * matrix [rows][cols] is cut into blocks of 32 consecutive elements of a row; a
 * block has one scale 2^e and each element is an E2M1 number (0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives) times that scale:
 *
 *   e = max(floor(log2(max |x|)) - 2, -127),   element = E2M1(x * 2^-e)
 *
 * rounded to nearest, ties to the even code, saturating at 6.  A block that
 * holds a NaN or an infinity reads as NaN throughout; a block of zeros as zeros.
 *
 * Memory, for rows x cols with B = ceil(cols/32) blocks to a row:
 *   data    [rows][16*B] bytes, element 2j of a row in the low half of byte j;
 *           elements past cols are zero.
 *   scales  one byte (e + 127; 255 = NaN) per block, in tiles of 128 rows x 4
 *           blocks = 512 bytes: row r, block b of a tile at
 *           16*(r % 32) + 4*((r % 128) / 32) + b % 4, tiles row-major, i.e.
 *           tile (r/128, b/4) at 512 * ((r/128) * ceil(B/4) + b/4).  Bytes of
 *           the tiles beyond the matrix are zero (the product needs that of the
 *           blocks past B).  One tile is what one copy moves into tensor memory.
 *
 * The conventions are conv2d.h's (status codes, caller-owned device memory, work
 * enqueued on `stream`, nothing allocated); data and scales are 16-byte aligned.
 */
#ifndef SPLIT_GEMM_GB300_MXFP4_H
#define SPLIT_GEMM_GB300_MXFP4_H

#include "conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of data and of scales for a matrix of rows x cols; 0 where either is below 1 or past 2^31 - 1. */
size_t mxfp4_data_bytes(int64_t rows, int64_t cols);
size_t mxfp4_scale_bytes(int64_t rows, int64_t cols);

/* Quantises x [rows][cols] (x_dtype: conv2d_out_dtype; x_stride elements from
 * one row to the next; aligned to its element type).  data/scales: of x, blocks
 * along its rows; data_t/scales_t: of the transpose [cols][rows], blocks along
 * x's columns.  Either pair may be NULL, not both; both come from one reading of x. */
int mxfp4_quantize(int64_t rows, int64_t cols, const void* x_dev, int32_t x_dtype, int64_t x_stride,
                   void* data_dev, void* scales_dev, void* data_t_dev, void* scales_t_dev,
                   conv2d_stream_t stream);

/* y [rows][cols], dense, of y_dtype: the values that data and scales stand for,
 * exact in fp32 and in bf16.  The quantiser's scale bytes are at most 252 (or
 * 255, NaN); with 253 and 254 from elsewhere the largest elements are past
 * either type and read as infinities. */
int mxfp4_dequantize(int64_t rows, int64_t cols, const void* data_dev, const void* scales_dev, void* y_dev,
                     int32_t y_dtype, conv2d_stream_t stream);

/* y[i][j] = act(sum_l a[i][l] * b[j][l] + bias[j]) for quantised a [m][k] and
 * b [n][k]; y [m][n] dense, of epi->out_dtype (fp32 when epi is NULL), act by
 * epi->activation.  Products are exact and sums are fp32; a sum split between
 * blocks is joined in a fixed order, so the same call gives the same bits.
 * bias_dev: [n] fp32 or NULL; y_dev is aligned to 16 bytes.  k = 0 is refused; m or n of 0
 * is an empty result. */
typedef struct {
    int64_t m, n, k;
} mxfp4_matmul_params;

int mxfp4_matmul(const mxfp4_matmul_params* params, const void* a_data_dev, const void* a_scales_dev,
                 const void* b_data_dev, const void* b_scales_dev, const float* bias_dev, void* y_dev,
                 const conv2d_epilogue* epi, conv2d_stream_t stream);

/* Synchronises `stream` and returns CONV2D_OK, or CONV2D_ERR_TIMEOUT if a
 * device-side wait (each is bounded, by seconds) ran out in any mxfp4_matmul on
 * the current device since the last time this was asked; that call's y is undefined then.
 * The device has one such word for all streams and threads: each report is told
 * once, to whoever asks first, so a program asks in one place and holds all of
 * its products since the last answer for undefined.  Threads may ask at the same time. */
int mxfp4_matmul_status(conv2d_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLIT_GEMM_GB300_MXFP4_H */
