// Layer normalisation kernels for rows of any width and alignment: the row is read
// again for each pass over it.  The fallback where a row does not fit the registers of a block (ln_rows.cuh).
// One element to a load, and L2 holds a row's second and third reading: 8192 x 16383 bf16 forward 209 us, backward 501 to 517.
#pragma once

#include "ln_params.cuh"
#include "ptx.cuh"

namespace sgb {
namespace ln {

constexpr int THREADS = 256;

// Sum over the block's threads, the same value (and the same order of additions) in all of them.
__device__ __forceinline__ float block_sum(float v, float* warp_sums)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // warp_sums may still be read from the previous sum
    if ((threadIdx.x & 31) == 0) warp_sums[warp] = v;
    __syncthreads();
    v = warp_sums[threadIdx.x & (THREADS / 32 - 1)];
#pragma unroll
    for (int o = THREADS / 64; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// mean and rstd of row x by the block: two readings, the second of the deviations' squares.
template <typename TX>
__device__ __forceinline__ void row_stats(const TX* x, const FwdParams& p, float* warp_sums, float& mean, float& rstd)
{
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += THREADS) s += mx::to_float(x[c]);
    mean = block_sum(s, warp_sums) * p.inv_cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += THREADS) {
        const float d = mx::to_float(x[c]) - mean;
        q = fmaf(d, d, q);
    }
    rstd = 1.f / sqrtf(block_sum(q, warp_sums) * p.inv_cols + p.eps);
}

__device__ __forceinline__ float normalised(float x, float mean, float rstd, const FwdParams& p, int c)
{
    const float w = p.weight ? p.weight[c] : 1.f, b = p.bias ? p.bias[c] : 0.f;
    return fmaf((x - mean) * rstd, w, b);
}

// One block per row, the row read three times.
template <typename TX, typename TY>
__global__ void __launch_bounds__(THREADS) fwd_any(const TX* x, TY* y, const FwdParams p)
{
    __shared__ float warp_sums[THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TX* xr = x + r * p.x_stride;
        float mean, rstd;
        row_stats(xr, p, warp_sums, mean, rstd);
        for (int c = threadIdx.x; c < p.cols; c += THREADS)
            mx::from_float(y[r * p.y_stride + c], normalised(mx::to_float(xr[c]), mean, rstd, p, c));
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// The same with a quantised result: a warp takes 32 columns, one block of the format, at a time.
template <typename TX>
__global__ void __launch_bounds__(THREADS) fwd_mx_any(const TX* x, const FwdParams p)
{
    __shared__ float warp_sums[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = mx::cdiv(p.cols, mx::BLOCK), btiles = mx::cdiv(blocks, mx::TILE_BLOCKS);
    for (int64_t r = blockIdx.x; r < p.padded_rows; r += gridDim.x) {
        if (r >= p.rows) {  // the scale tiles' padding rows
            for (int b = threadIdx.x; b < btiles * mx::TILE_BLOCKS; b += THREADS) p.scales[mx::scale_at(r, b, btiles)] = 0;
            continue;
        }
        const TX* xr = x + r * p.x_stride;
        float mean, rstd;
        row_stats(xr, p, warp_sums, mean, rstd);
        for (int b = warp; b < btiles * mx::TILE_BLOCKS; b += THREADS / 32) {
            const int c = b * mx::BLOCK + lane;
            const float v = c < p.cols ? normalised(mx::to_float(xr[c]), mean, rstd, p, c) : 0.f;
            const uint32_t byte = mx::scale_byte(__reduce_max_sync(0xffffffffu, mx::abs_bits(v)));
            if (lane == 0) p.scales[mx::scale_at(r, b, btiles)] = static_cast<uint8_t>(byte);
            if (b >= blocks) continue;
            const float q = v * mx::inverse_scale(byte);
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = __shfl_sync(0xffffffffu, q, 8 * (lane & 3) + j);
            const uint32_t word = mx::pack_e2m1x8(e);
            if (lane < 4) *reinterpret_cast<uint32_t*>(p.data + (r * blocks + b) * 16 + 4 * lane) = word;
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// dx, one block per row, the row read twice.
template <typename TX, typename TY>
__global__ void __launch_bounds__(THREADS) bwd_dx_any(const TY* dy, const TX* x, TX* dx, const BwdParams p)
{
    __shared__ float warp_sums[THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TX* xr = x + r * p.x_stride;
        const TY* dyr = dy + r * p.dy_stride;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            s1 += g;
            s2 = fmaf(g, (mx::to_float(xr[c]) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, warp_sums) * p.inv_cols;
        s2 = block_sum(s2, warp_sums) * p.inv_cols;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            const float xh = (mx::to_float(xr[c]) - mean) * rstd;
            mx::from_float(dx[r * p.cols + c], rstd * (g - s1 - xh * s2));
        }
    }
}

// Partial sums of dweight and dbias for rows too wide for registers: a thread keeps VEC columns and takes every
// p.chunks-th row.  Rows of one part lie a multiple of 8 rows apart, so they begin at the same place within 16 bytes, and vectors
// are whole from there: what stands in front of a row (the row before) adds to sums that are not written.  Bound by HBM.
template <typename TX, typename TY, int VEC>
__global__ void __launch_bounds__(THREADS) bwd_part_any(const TY* __restrict__ dy, const TX* __restrict__ x, const BwdParams p)
{
    const int k = blockIdx.y;
    const int off = VEC > 1 ? static_cast<int>(k * p.x_stride % VEC) : 0;
    const int c0 = (blockIdx.x * THREADS + threadIdx.x) * VEC - off;
    if (c0 >= p.cols) return;
    const bool tail = c0 + VEC > p.cols;  // the last row's end may be the tensor's
    float dw[VEC] = {}, db[VEC] = {};
#pragma unroll 4
    for (int64_t r = k; r < p.rows; r += p.chunks) {
        const float mean = __ldg(p.mean + r), rstd = __ldg(p.rstd + r);
        const TX* xr = x + r * p.x_stride + c0;
        const TY* gr = dy + r * p.dy_stride + c0;
        struct alignas(sizeof(TX) * VEC < 16 ? sizeof(TX) * VEC : 16) X { TX v[VEC]; } xv;
        struct alignas(sizeof(TY) * VEC < 16 ? sizeof(TY) * VEC : 16) G { TY v[VEC]; } gv;
        if (!tail) {
            xv = *reinterpret_cast<const X*>(xr);
            gv = *reinterpret_cast<const G*>(gr);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const bool in = c0 + i >= 0 && c0 + i < p.cols;
                xv.v[i] = in ? xr[i] : TX(0.f);
                gv.v[i] = in ? gr[i] : TY(0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float g = mx::to_float(gv.v[i]);
            dw[i] = fmaf(g, (mx::to_float(xv.v[i]) - mean) * rstd, dw[i]);
            db[i] += g;
        }
    }
    float* part = p.part + 2 * static_cast<int64_t>(k) * p.cols;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (c0 + i >= 0 && c0 + i < p.cols) {
            part[c0 + i] = dw[i];
            part[p.cols + c0 + i] = db[i];
        }
}

// Joins the partial sums in a fixed order: a block has 32 columns and 32 sums of every 32nd part.
static __global__ void __launch_bounds__(1024) bwd_join(const BwdParams p)
{
    __shared__ float sums[2][32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    float dw = 0.f, db = 0.f;
    ptx::grid_dependency_wait();  // started early
    if (c < p.cols)
        for (int k = ty; k < p.chunks; k += 32) {
            dw += p.part[(2 * static_cast<int64_t>(k)) * p.cols + c];
            db += p.part[(2 * static_cast<int64_t>(k) + 1) * p.cols + c];
        }
    sums[0][tx][ty] = dw;
    sums[1][tx][ty] = db;
    __syncthreads();
    // warp ty sums column ty's 32 values, lane by lane
    dw = sums[0][ty][tx];
    db = sums[1][ty][tx];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        dw += __shfl_xor_sync(0xffffffffu, dw, o);
        db += __shfl_xor_sync(0xffffffffu, db, o);
    }
    const int out = blockIdx.x * 32 + ty;
    if (tx == 0 && out < p.cols) {
        if (p.dweight) p.dweight[out] = dw;
        if (p.dbias) p.dbias[out] = db;
    }
}

inline int join_parts(const BwdParams& p, cudaStream_t stream)
{
    return mx::launch(bwd_join, mx::cdiv(p.cols, 32), 1024, 0, stream, 1, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

}  // namespace ln
}  // namespace sgb
