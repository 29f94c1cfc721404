// The product of two microscaled 4-bit matrices: host side and kernels.
#include "mxfp4.h"

#include "mx_common.cuh"

namespace sgb {
namespace mx {

struct ProductParams {
    int64_t m, n, k, blocks, btiles;
    const uint8_t *a, *a_scales, *b, *b_scales;
    const float* bias;
    int relu;
};

constexpr int P_TILE = 64;

// y = relu?(a b^T + bias) in fp32 multiply-adds: a 64 x 64 tile per block of
// threads, one block of 32 along the reduction at a time.
template <typename T>
__global__ void __launch_bounds__(256) product_kernel(T* y, const ProductParams p)
{
    __shared__ float a[P_TILE][BLOCK + 1], b[P_TILE][BLOCK + 1];
    const int64_t ntiles = cdiv<int64_t>(p.n, P_TILE);
    const int64_t m0 = blockIdx.x / ntiles * P_TILE, n0 = blockIdx.x % ntiles * P_TILE;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t kb = 0; kb < p.blocks; ++kb) {
        const int i = threadIdx.x >> 2, w = threadIdx.x & 3;  // row of the tile, word of the block
        const int64_t ra = m0 + i, rb = n0 + i;
        const uint32_t wa = ra < p.m ? *reinterpret_cast<const uint32_t*>(p.a + (ra * p.blocks + kb) * 16 + 4 * w) : 0u;
        const uint32_t wb = rb < p.n ? *reinterpret_cast<const uint32_t*>(p.b + (rb * p.blocks + kb) * 16 + 4 * w) : 0u;
        const float sa = ra < p.m ? scale_value(p.a_scales[scale_at(ra, kb, p.btiles)]) : 0.f;
        const float sb = rb < p.n ? scale_value(p.b_scales[scale_at(rb, kb, p.btiles)]) : 0.f;
        for (int j = 0; j < 8; ++j) {
            a[i][8 * w + j] = e2m1_value(wa >> (4 * j) & 15u) * sa;
            b[i][8 * w + j] = e2m1_value(wb >> (4 * j) & 15u) * sb;
        }
        __syncthreads();
        for (int k = 0; k < BLOCK; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(a[ty + 16 * u][k], b[tx + 16 * v][k], acc[u][v]);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t r = m0 + ty + 16 * u, c = n0 + tx + 16 * v;
            if (r >= p.m || c >= p.n) continue;
            float s = acc[u][v] + (p.bias ? p.bias[c] : 0.f);
            if (p.relu && !(s > 0.f) && s == s) s = 0.f;  // NaN stays
            from_float(y[r * p.n + c], s);
        }
}

}  // namespace mx
}  // namespace sgb

using namespace sgb;

extern "C" int mxfp4_matmul(const mxfp4_matmul_params* params, const void* a_data_dev, const void* a_scales_dev,
                            const void* b_data_dev, const void* b_scales_dev, const float* bias_dev, void* y_dev,
                            const conv2d_epilogue* epi, conv2d_stream_t stream)
{
    constexpr int64_t most = (int64_t(1) << 31) - 1;
    if (!params || params->m < 0 || params->n < 0 || params->k < 1) return CONV2D_ERR_INVALID;
    if (params->m > most || params->n > most || params->k > most) return CONV2D_ERR_UNSUPPORTED;
    const int act = epi ? epi->activation : CONV2D_ACT_NONE, out = epi ? epi->out_dtype : CONV2D_OUT_F32;
    if ((act != CONV2D_ACT_NONE && act != CONV2D_ACT_RELU) || (out != CONV2D_OUT_F32 && out != CONV2D_OUT_BF16))
        return CONV2D_ERR_INVALID;
    if (params->m == 0 || params->n == 0) return CONV2D_OK;
    if (!a_data_dev || !a_scales_dev || !b_data_dev || !b_scales_dev || !y_dev) return CONV2D_ERR_INVALID;
    for (const void* p : {a_data_dev, a_scales_dev, b_data_dev, b_scales_dev, static_cast<const void*>(y_dev)})
        if (reinterpret_cast<uintptr_t>(p) % 16) return CONV2D_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(bias_dev) % 4) return CONV2D_ERR_ALIGNMENT;
    mx::ProductParams k{};
    k.m = params->m;
    k.n = params->n;
    k.k = params->k;
    k.blocks = mx::cdiv<int64_t>(k.k, mx::BLOCK);
    k.btiles = mx::cdiv<int64_t>(k.blocks, mx::TILE_BLOCKS);
    k.a = static_cast<const uint8_t*>(a_data_dev);
    k.a_scales = static_cast<const uint8_t*>(a_scales_dev);
    k.b = static_cast<const uint8_t*>(b_data_dev);
    k.b_scales = static_cast<const uint8_t*>(b_scales_dev);
    k.bias = bias_dev;
    k.relu = act == CONV2D_ACT_RELU;
    const int64_t grid = mx::cdiv<int64_t>(k.m, mx::P_TILE) * mx::cdiv<int64_t>(k.n, mx::P_TILE);
    if (grid > most) return CONV2D_ERR_UNSUPPORTED;
    if (out == CONV2D_OUT_BF16)
        mx::product_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(static_cast<__nv_bfloat16*>(y_dev), k);
    else
        mx::product_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(static_cast<float*>(y_dev), k);
    return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}
