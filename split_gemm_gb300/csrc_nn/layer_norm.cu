// Layer normalisation forward and backward: host side and the kernels for rows of any width.
#include "layer_norm.h"

#include "mxfp4.h"
#include "mx_common.cuh"

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

struct FwdParams {
    int64_t rows, x_stride, y_stride, padded_rows;
    int cols;
    float eps, inv_cols;
    const float *weight, *bias;
    float *mean, *rstd;
    uint8_t *data, *scales;
};

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

struct BwdParams {
    int64_t rows, x_stride, dy_stride, chunk;
    int cols;
    float inv_cols;
    const float *mean, *rstd, *weight;
    float *dweight, *dbias, *part;  // part: [chunks][2][cols]
    int chunks;
};

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

// Partial sums of dweight and dbias over one chunk of rows, a thread to a column.
template <typename TX, typename TY>
__global__ void __launch_bounds__(THREADS) bwd_part_any(const TY* dy, const TX* x, const BwdParams p)
{
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= p.cols) return;
    for (int k = blockIdx.y; k < p.chunks; k += gridDim.y) {
        const int64_t r0 = k * p.chunk, r1 = r0 + p.chunk < p.rows ? r0 + p.chunk : p.rows;
        float dw = 0.f, db = 0.f;
        for (int64_t r = r0; r < r1; ++r) {
            const float g = mx::to_float(dy[r * p.dy_stride + c]);
            dw = fmaf(g, (mx::to_float(x[r * p.x_stride + c]) - p.mean[r]) * p.rstd[r], dw);
            db += g;
        }
        p.part[(2 * static_cast<int64_t>(k)) * p.cols + c] = dw;
        p.part[(2 * static_cast<int64_t>(k) + 1) * p.cols + c] = db;
    }
}

// Joins the partial sums, in the chunks' order.
__global__ void __launch_bounds__(THREADS) bwd_join(const BwdParams p)
{
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= p.cols) return;
    float dw = 0.f, db = 0.f;
    for (int k = 0; k < p.chunks; ++k) {
        dw += p.part[(2 * static_cast<int64_t>(k)) * p.cols + c];
        db += p.part[(2 * static_cast<int64_t>(k) + 1) * p.cols + c];
    }
    if (p.dweight) p.dweight[c] = dw;
    if (p.dbias) p.dbias[c] = db;
}

// ---------------------------------------------------------------- host
constexpr int64_t MAX_ROWS = (int64_t(1) << 31) - 1;
constexpr int64_t MAX_COLS = int64_t(1) << 30;  // column counters are ints and step past the end

bool dtype_ok(int32_t t) { return t == CONV2D_OUT_F32 || t == CONV2D_OUT_BF16; }
size_t dtype_size(int32_t t) { return t == CONV2D_OUT_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check(const layer_norm_params* p, bool y)
{
    if (!p || p->rows < 0 || p->cols < 1) return CONV2D_ERR_INVALID;
    if (p->rows > MAX_ROWS || p->cols > MAX_COLS) return CONV2D_ERR_UNSUPPORTED;
    if (!dtype_ok(p->x_dtype) || p->x_stride < p->cols || !(p->eps >= 0.f)) return CONV2D_ERR_INVALID;
    if (y && (!dtype_ok(p->y_dtype) || p->y_stride < p->cols)) return CONV2D_ERR_INVALID;
    return CONV2D_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA; }

unsigned row_grid(int64_t rows) { return static_cast<unsigned>(rows < 65536 ? rows : 65536); }

FwdParams fwd_params(const layer_norm_params* p, const float* weight, const float* bias, float* mean, float* rstd)
{
    FwdParams k{};
    k.rows = p->rows;
    k.x_stride = p->x_stride;
    k.y_stride = p->y_stride;
    k.padded_rows = mx::cdiv<int64_t>(p->rows, mx::TILE_ROWS) * mx::TILE_ROWS;
    k.cols = static_cast<int>(p->cols);
    k.eps = p->eps;
    k.inv_cols = 1.f / static_cast<float>(p->cols);
    k.weight = weight;
    k.bias = bias;
    k.mean = mean;
    k.rstd = rstd;
    return k;
}

// Calls f with null pointers of the two element types.
template <typename F>
void by_types(int32_t x, int32_t y, F&& f)
{
    float* f32 = nullptr;
    __nv_bfloat16* b16 = nullptr;
    if (x == CONV2D_OUT_BF16)
        y == CONV2D_OUT_BF16 ? f(b16, b16) : f(b16, f32);
    else
        y == CONV2D_OUT_BF16 ? f(f32, b16) : f(f32, f32);
}

constexpr int64_t PART_ROWS = 64;    // rows of one chunk, at least
constexpr int64_t PART_CHUNKS = 512;  // chunks, at most

int64_t part_chunks(int64_t rows)
{
    const int64_t n = mx::cdiv(rows, PART_ROWS);
    return n < PART_CHUNKS ? n : PART_CHUNKS;
}

}  // namespace ln
}  // namespace sgb

using namespace sgb;

extern "C" int layer_norm_fwd(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                              const float* bias_dev, void* y_dev, float* mean_dev, float* rstd_dev,
                              conv2d_stream_t stream)
{
    if (int rc = ln::check(params, true)) return rc;
    if (params->rows == 0) return CONV2D_OK;
    if (!x_dev || !y_dev) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(y_dev, ln::dtype_size(params->y_dtype)) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(bias_dev, 4) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4))
        return CONV2D_ERR_ALIGNMENT;
    const ln::FwdParams k = ln::fwd_params(params, weight_dev, bias_dev, mean_dev, rstd_dev);
    ln::by_types(params->x_dtype, params->y_dtype, [&](auto* tx, auto* ty) {
        ln::fwd_any<<<ln::row_grid(k.rows), ln::THREADS, 0, stream>>>(static_cast<decltype(tx)>(const_cast<void*>(x_dev)),
                                                                     static_cast<decltype(ty)>(y_dev), k);
    });
    return ln::launched();
}

extern "C" int layer_norm_mxfp4(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                                const float* bias_dev, void* data_dev, void* scales_dev, float* mean_dev,
                                float* rstd_dev, conv2d_stream_t stream)
{
    if (int rc = ln::check(params, false)) return rc;
    if (params->rows == 0) return CONV2D_OK;
    if (!x_dev || !data_dev || !scales_dev) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(data_dev, 16) || !ln::aligned(scales_dev, 16) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(bias_dev, 4) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4))
        return CONV2D_ERR_ALIGNMENT;
    ln::FwdParams k = ln::fwd_params(params, weight_dev, bias_dev, mean_dev, rstd_dev);
    k.data = static_cast<uint8_t*>(data_dev);
    k.scales = static_cast<uint8_t*>(scales_dev);
    ln::by_types(params->x_dtype, CONV2D_OUT_F32, [&](auto* tx, auto*) {
        ln::fwd_mx_any<<<ln::row_grid(k.padded_rows), ln::THREADS, 0, stream>>>(
            static_cast<decltype(tx)>(const_cast<void*>(x_dev)), k);
    });
    return ln::launched();
}

extern "C" size_t layer_norm_bwd_workspace_bytes(const layer_norm_params* params)
{
    if (ln::check(params, true)) return 0;
    return static_cast<size_t>(ln::part_chunks(params->rows)) * 2 * static_cast<size_t>(params->cols) * sizeof(float);
}

extern "C" int layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* x_dev,
                              const float* mean_dev, const float* rstd_dev, const float* weight_dev, void* dx_dev,
                              float* dweight_dev, float* dbias_dev, void* workspace_dev, size_t workspace_bytes,
                              conv2d_stream_t stream)
{
    if (int rc = ln::check(params, true)) return rc;
    const bool sums = dweight_dev || dbias_dev;
    if (params->rows > 0 && (!dy_dev || !x_dev || !mean_dev || !rstd_dev || !dx_dev)) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(dx_dev, ln::dtype_size(params->x_dtype)) ||
        !ln::aligned(dy_dev, ln::dtype_size(params->y_dtype)) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(dweight_dev, 4) || !ln::aligned(dbias_dev, 4) || !ln::aligned(workspace_dev, 16))
        return CONV2D_ERR_ALIGNMENT;
    const size_t need = layer_norm_bwd_workspace_bytes(params);
    if (sums && need && (!workspace_dev || workspace_bytes < need)) return CONV2D_ERR_WORKSPACE;
    ln::BwdParams k{};
    k.rows = params->rows;
    k.x_stride = params->x_stride;
    k.dy_stride = params->y_stride;
    k.cols = static_cast<int>(params->cols);
    k.inv_cols = 1.f / static_cast<float>(params->cols);
    k.mean = mean_dev;
    k.rstd = rstd_dev;
    k.weight = weight_dev;
    k.dweight = dweight_dev;
    k.dbias = dbias_dev;
    k.part = static_cast<float*>(workspace_dev);
    k.chunks = static_cast<int>(ln::part_chunks(params->rows));
    k.chunk = k.chunks ? mx::cdiv<int64_t>(params->rows, k.chunks) : 0;
    const unsigned col_grid = static_cast<unsigned>(mx::cdiv(k.cols, ln::THREADS));
    if (params->rows > 0)
        ln::by_types(params->x_dtype, params->y_dtype, [&](auto* tx, auto* ty) {
            auto* x = static_cast<decltype(tx)>(const_cast<void*>(x_dev));
            auto* dy = static_cast<decltype(ty)>(const_cast<void*>(dy_dev));
            ln::bwd_dx_any<<<ln::row_grid(k.rows), ln::THREADS, 0, stream>>>(dy, x, static_cast<decltype(tx)>(dx_dev), k);
            if (sums) ln::bwd_part_any<<<dim3(col_grid, k.chunks), ln::THREADS, 0, stream>>>(dy, x, k);
        });
    if (sums) ln::bwd_join<<<col_grid, ln::THREADS, 0, stream>>>(k);
    return ln::launched();
}
