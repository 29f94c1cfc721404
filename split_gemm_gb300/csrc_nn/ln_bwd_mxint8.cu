// The norm's gradient with x as an 8-bit checkpoint (mxint8.h).
#include "mxint8.h"

#include "ln_any.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ln {

// A checkpoint's rows.
struct Checkpoint {
    const uint8_t *data, *scales;
    int64_t blocks;
    __device__ __forceinline__ float at(int64_t r, int64_t c) const
    {
        const int q = static_cast<int8_t>(__ldg(data + r * (blocks * mx::BLOCK) + c));
        return static_cast<float>(q) * 0.015625f * mx::scale_value(__ldg(scales + r * blocks + c / mx::BLOCK));
    }
};

// dx, one block per row, the row read twice: the form for rows of any width and alignment.
template <typename TY>
__global__ void __launch_bounds__(THREADS) bwd8_dx_any(const TY* dy, const Checkpoint x, TY* dx, const BwdParams p)
{
    __shared__ float warp_sums[THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TY* dyr = dy + r * p.dy_stride;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            s1 += g;
            s2 = fmaf(g, (x.at(r, c) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, warp_sums) * p.inv_cols;
        s2 = block_sum(s2, warp_sums) * p.inv_cols;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            const float xh = (x.at(r, c) - mean) * rstd;
            mx::from_float(dx[r * p.cols + c], rstd * (g - s1 - xh * s2));
        }
    }
}

// Partial sums of dweight and dbias: a thread keeps its column and takes every p.chunks-th row.
template <typename TY>
__global__ void __launch_bounds__(THREADS) bwd8_part_any(const TY* __restrict__ dy, const Checkpoint x, const BwdParams p)
{
    const int64_t c = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
    if (c >= p.cols) return;
    float dw = 0.f, db = 0.f;
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < p.rows; r += p.chunks) {
        const float g = mx::to_float(dy[r * p.dy_stride + c]);
        dw = fmaf(g, (x.at(r, c) - __ldg(p.mean + r)) * __ldg(p.rstd + r), dw);
        db += g;
    }
    float* part = p.part + 2 * static_cast<int64_t>(blockIdx.y) * p.cols;
    part[c] = dw;
    part[p.cols + c] = db;
}

constexpr int64_t ANY_PART_ROWS = 32, ANY_PARTS = 128;

int64_t bwd8_parts(const layer_norm_params* p)
{
    const int64_t n = mx::cdiv(p->rows, ANY_PART_ROWS);
    return n < ANY_PARTS ? n : ANY_PARTS;
}

int check8(const layer_norm_params* p)
{
    constexpr int64_t most_rows = (int64_t(1) << 31) - 32, most_cols = int64_t(1) << 30;
    if (!p || p->rows < 0 || p->cols < 1) return CONV2D_ERR_INVALID;
    if (p->rows > most_rows || p->cols > most_cols) return CONV2D_ERR_UNSUPPORTED;
    if ((p->y_dtype != CONV2D_OUT_F32 && p->y_dtype != CONV2D_OUT_BF16) || p->y_stride < p->cols) return CONV2D_ERR_INVALID;
    return CONV2D_OK;
}

template <typename TY>
int bwd8(const BwdParams& k, const Checkpoint& x, cudaStream_t stream)
{
    const TY* dy = static_cast<const TY*>(k.dy);
    const unsigned grid = static_cast<unsigned>(k.rows < 65536 ? k.rows : 65536);
    bwd8_dx_any<<<grid, THREADS, 0, stream>>>(dy, x, static_cast<TY*>(k.dx), k);
    if (k.part) {
        const dim3 parts(static_cast<unsigned>(mx::cdiv<int64_t>(k.cols, THREADS)), static_cast<unsigned>(k.chunks));
        bwd8_part_any<<<parts, THREADS, 0, stream>>>(dy, x, k);
    }
    return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

}  // namespace ln
}  // namespace sgb

using namespace sgb;

extern "C" size_t mxint8_layer_norm_bwd_workspace_bytes(const layer_norm_params* params)
{
    if (ln::check8(params)) return 0;
    return static_cast<size_t>(ln::bwd8_parts(params)) * 2 * static_cast<size_t>(params->cols) * sizeof(float);
}

extern "C" int mxint8_layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* data_dev, const void* scales_dev,
                                     const float* mean_dev, const float* rstd_dev, const float* weight_dev, void* dx_dev,
                                     float* dweight_dev, float* dbias_dev, void* workspace_dev, size_t workspace_bytes,
                                     conv2d_stream_t stream)
{
    if (int rc = ln::check8(params)) return rc;
    const bool sums = dweight_dev || dbias_dev;
    if (params->rows > 0 && (!dy_dev || !data_dev || !scales_dev || !mean_dev || !rstd_dev || !dx_dev)) return CONV2D_ERR_INVALID;
    const auto aligned = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const size_t sy = params->y_dtype == CONV2D_OUT_BF16 ? 2 : 4;
    if (!aligned(data_dev, 16) || !aligned(dx_dev, sy) || !aligned(dy_dev, sy) || !aligned(mean_dev, 4) || !aligned(rstd_dev, 4) ||
        !aligned(weight_dev, 4) || !aligned(dweight_dev, 4) || !aligned(dbias_dev, 4) || !aligned(workspace_dev, 16))
        return CONV2D_ERR_ALIGNMENT;
    const size_t need = mxint8_layer_norm_bwd_workspace_bytes(params);
    if (sums && need && (!workspace_dev || workspace_bytes < need)) return CONV2D_ERR_WORKSPACE;
    ln::BwdParams k{};
    k.rows = params->rows;
    k.dy_stride = params->y_stride;
    k.cols = static_cast<int>(params->cols);
    k.inv_cols = 1.f / static_cast<float>(params->cols);
    k.mean = mean_dev;
    k.rstd = rstd_dev;
    k.weight = weight_dev;
    k.dweight = dweight_dev;
    k.dbias = dbias_dev;
    k.dy = dy_dev;
    k.dx = dx_dev;
    k.part = sums ? static_cast<float*>(workspace_dev) : nullptr;
    k.chunks = static_cast<int>(ln::bwd8_parts(params));
    const ln::Checkpoint x{static_cast<const uint8_t*>(data_dev), static_cast<const uint8_t*>(scales_dev),
                           mx::cdiv<int64_t>(params->cols, mx::BLOCK)};
    int rc = CONV2D_OK;
    if (params->rows > 0) rc = params->y_dtype == CONV2D_OUT_BF16 ? ln::bwd8<__nv_bfloat16>(k, x, stream) : ln::bwd8<float>(k, x, stream);
    if (rc || !sums) return rc;
    return ln::join_parts(k, stream);
}
