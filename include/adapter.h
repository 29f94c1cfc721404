/*
 * adapter.h -- C ABI of low-rank adapters beside a shared projection: each row
 * of x (a token, or a pixel of NHWC activations) has one of many adapters, or none.
 *
 *   h[t]   = scale[e] * a[e] x[t]                       e = index[t]
 *   out[t] = act(y[t] + b[e] h[t])                      y: the shared projection's result
 *
 * and for an output gradient dy (after act's derivative, where there was one):
 *
 *   dh[t] = scale[e] * b[e]^T dy[t]
 *   dx[t] = dx0[t] + a[e]^T dh[t]                       dx0: the shared projection's part
 *   da[e] = sum over the rows t of e: dh[t] x[t]^T
 *   db[e] = sum over the rows t of e: dy[t] h[t]^T
 *
 * A row whose index is not in 0 .. adapters-1 has no adapter: out = act(y), dx = dx0,
 * h = 0, and it is in no sum; an adapter without rows gets zero gradients.  Rows of an
 * adapter may lie anywhere and in any order; adapters of lower rank are padded with zeros.
 *
 * x, a, b and dy are bf16, h and dh fp32.  Products of bf16 numbers are exact and their
 * sums fp32; h and dh enter their products as three bf16 parts that add up to all their 24 bits (down to 2^-110).
 * Where a row meets an infinity or a NaN in its own x, dy, h, a[e] or b[e], the sums they enter are not finite, NaN wherever
 * one of the parts is zero; they stay within that row, or that adapter's gradients.
 * A value is rounded once, where it is stored.  Sums over rows are joined in a fixed order:
 * the same call gives the same bits.
 *
 * The conventions are conv2d.h's (status codes, caller-owned device memory, work
 * enqueued on `stream`, nothing allocated), except that a pointer need only be aligned to its own element
 * type; rows of whole 16-byte vectors are read faster.
 */
#ifndef SPLIT_GEMM_GB300_ADAPTER_H
#define SPLIT_GEMM_GB300_ADAPTER_H

#include "conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A plan says where each adapter's rows are.  It depends on the index alone: a program makes it once for a batch and uses
 * it beside every layer, in any number of calls at once.  Bytes of device memory for it (0 where rows or
 * adapters are out of range: 0 <= rows < 2^31 - 2^16, 1 <= adapters <= 65535). */
size_t adapter_plan_bytes(int64_t rows, int64_t adapters);

/* index: [rows] int32.  plan_dev: adapter_plan_bytes() bytes of any content, 16-byte aligned. */
int adapter_plan(int64_t rows, int64_t adapters, const int32_t* index_dev, void* plan_dev, conv2d_stream_t stream);

typedef struct {
    int64_t rows, cols, outs;      /* x [rows][cols], y and out [rows][outs]; cols and outs from 1 to 2^30 */
    int64_t rank, adapters;        /* a [adapters][rank][cols], b [adapters][outs][rank], dense; rank from 1 to 128 */
    int64_t x_stride, y_stride, out_stride; /* elements from one row to the next, >= the row */
    int32_t y_dtype, out_dtype;    /* conv2d_out_dtype */
    int32_t activation;            /* conv2d_activation */
} adapter_fwd_params;

/* out may be y itself when type and stride are the same, and overlaps no other operand.  scale_dev: [adapters] fp32 or NULL (ones).
 * h_dev: [rows][rank] fp32, dense, for the backward pass; may be NULL.  plan_dev: of the same rows and adapters. */
int adapter_fwd(const adapter_fwd_params* params, const void* plan_dev, const void* y_dev, const void* x_dev,
                const void* a_dev, const void* b_dev, const float* scale_dev, void* out_dev, float* h_dev,
                conv2d_stream_t stream);

enum { ADAPTER_X_BF16 = 1, ADAPTER_X_MXINT8 = 2 };

typedef struct {
    int64_t rows, cols, outs, rank, adapters;
    int64_t dy_stride, x_stride, dx0_stride, dx_stride; /* x_stride: of bf16 x; an MXINT8 x is dense (mxint8.h) */
    int32_t x_type;                /* ADAPTER_X_BF16 or ADAPTER_X_MXINT8 */
    int32_t dx0_dtype, dx_dtype;   /* conv2d_out_dtype */
} adapter_bwd_params;

/* dx_dev, da_dev, db_dev: each may be NULL (not computed).  dx0_dev may be NULL (zeros), or dx itself when type and stride are
 * the same; no result overlaps another operand.  da [adapters][rank][cols] and db [adapters][outs][rank] fp32, dense.  x_dev (with x_scales_dev for MXINT8) is needed
 * for da, h_dev of the forward pass for db.  workspace_dev: at least
 * adapter_bwd_workspace_bytes() bytes of any content, 16-byte aligned. */
size_t adapter_bwd_workspace_bytes(const adapter_bwd_params* params);

int adapter_bwd(const adapter_bwd_params* params, const void* plan_dev, const void* dy_dev, const void* x_dev,
                const void* x_scales_dev, const float* h_dev, const void* a_dev, const void* b_dev,
                const float* scale_dev, const void* dx0_dev, void* dx_dev, float* da_dev, float* db_dev,
                void* workspace_dev, size_t workspace_bytes, conv2d_stream_t stream);

/* Synchronises `stream` and returns CONV2D_OK, or CONV2D_ERR_TIMEOUT if a device-side wait (each is bounded, by
 * seconds) ran out in any adapter call on the current device since the last time this was asked; that call's results
 * are undefined then.  The conventions are mxfp4_matmul_status()'s. */
int adapter_status(conv2d_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLIT_GEMM_GB300_ADAPTER_H */
