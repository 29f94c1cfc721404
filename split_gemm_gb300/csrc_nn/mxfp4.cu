// Microscaled 4-bit matrices: quantisation by rows, by columns or both, and the way back.
#include "mxfp4.h"

#include "mx_common.cuh"

namespace sgb {
namespace mx {

constexpr int64_t MAX_EXTENT = (int64_t(1) << 31) - 1;

bool extents_ok(int64_t rows, int64_t cols) { return rows >= 1 && cols >= 1 && rows <= MAX_EXTENT && cols <= MAX_EXTENT; }

struct QuantParams {
    int64_t rows, cols, x_stride;
    int64_t row_tiles, col_tiles;  // of 128 x 128 elements
    uint8_t *data, *scales, *data_t, *scales_t;
};

// A block of threads takes a tile of 128 x 128 elements, which is one scale tile
// of either form.  A warp quantises one block of 32 at a time, a lane to an element.
constexpr int Q_TILE = 128;
constexpr int Q_THREADS = 256;

// Quantises the lanes' values as one block: returns the block's scale byte in
// every lane and, in lanes 0..3, the words of its 16 bytes.
__device__ __forceinline__ uint32_t quantize_warp(float v, uint32_t& word)
{
    const int lane = threadIdx.x & 31;
    const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(v)));
    const float q = v * inverse_scale(byte);
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = __shfl_sync(0xffffffffu, q, 8 * (lane & 3) + j);
    word = pack_e2m1x8(e);
    return byte;
}

template <typename T>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(const T* x, const QuantParams p)
{
    __shared__ float tile[Q_TILE][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rb = blockIdx.x / p.col_tiles, cb = blockIdx.x % p.col_tiles;
    const int64_t row_blocks = cdiv<int64_t>(p.rows, BLOCK), col_blocks = cdiv<int64_t>(p.cols, BLOCK);
    for (int b = 0; b < TILE_BLOCKS; ++b) {  // 32 columns at a time
        const int64_t kb = cb * TILE_BLOCKS + b;
        const int64_t c = kb * BLOCK + lane;
        for (int i = warp; i < Q_TILE; i += Q_THREADS / 32) {
            const int64_t r = rb * Q_TILE + i;
            const float v = r < p.rows && c < p.cols ? to_float(x[r * p.x_stride + c]) : 0.f;
            tile[i][lane] = v;
            if (!p.data) continue;
            uint32_t word;
            const uint32_t byte = quantize_warp(v, word);
            if (lane == 0) p.scales[scale_at(r, kb, p.col_tiles)] = static_cast<uint8_t>(byte);
            if (r < p.rows && kb < col_blocks && lane < 4)
                *reinterpret_cast<uint32_t*>(p.data + (r * col_blocks + kb) * 16 + 4 * lane) = word;
        }
        __syncthreads();
        if (p.data_t) {
            for (int i = warp; i < 32 * TILE_BLOCKS; i += Q_THREADS / 32) {
                const int col = i & 31, g = i >> 5;
                uint32_t word;
                const uint32_t byte = quantize_warp(tile[g * BLOCK + lane][col], word);
                const int64_t r = kb * BLOCK + col, k = rb * TILE_BLOCKS + g;  // row and block of the transpose
                if (lane == 0) p.scales_t[scale_at(r, k, p.row_tiles)] = static_cast<uint8_t>(byte);
                if (r < p.cols && k < row_blocks && lane < 4)
                    *reinterpret_cast<uint32_t*>(p.data_t + (r * row_blocks + k) * 16 + 4 * lane) = word;
            }
        }
        __syncthreads();
    }
}

// A thread takes 8 elements: 4 bytes in, 16 or 32 out.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* data, const uint8_t* scales, T* y, int64_t rows,
                                                         int64_t cols)
{
    const int64_t blocks = cdiv<int64_t>(cols, BLOCK), btiles = cdiv<int64_t>(blocks, TILE_BLOCKS);
    const int64_t n = rows * blocks * 4;
    for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / (blocks * 4), w = i - r * (blocks * 4);
        const uint32_t word = reinterpret_cast<const uint32_t*>(data)[i];
        const float s = scale_value(scales[scale_at(r, w >> 2, btiles)]);
        for (int j = 0; j < 8; ++j) {
            const int64_t c = w * 8 + j;
            if (c < cols) from_float(y[r * cols + c], e2m1_value(word >> (4 * j) & 15u) * s);
        }
    }
}

}  // namespace mx
}  // namespace sgb

using namespace sgb;

extern "C" size_t mxfp4_data_bytes(int64_t rows, int64_t cols)
{
    if (!mx::extents_ok(rows, cols)) return 0;
    return static_cast<size_t>(rows) * static_cast<size_t>(mx::cdiv<int64_t>(cols, mx::BLOCK)) * 16;
}

extern "C" size_t mxfp4_scale_bytes(int64_t rows, int64_t cols)
{
    if (!mx::extents_ok(rows, cols)) return 0;
    return static_cast<size_t>(mx::cdiv<int64_t>(rows, mx::TILE_ROWS)) *
           static_cast<size_t>(mx::cdiv<int64_t>(cols, mx::BLOCK * mx::TILE_BLOCKS)) * mx::TILE_BYTES;
}

extern "C" int mxfp4_quantize(int64_t rows, int64_t cols, const void* x_dev, int32_t x_dtype, int64_t x_stride,
                              void* data_dev, void* scales_dev, void* data_t_dev, void* scales_t_dev,
                              conv2d_stream_t stream)
{
    if (rows < 0 || cols < 1 || x_stride < cols || (x_dtype != CONV2D_OUT_F32 && x_dtype != CONV2D_OUT_BF16))
        return CONV2D_ERR_INVALID;
    if (!data_dev != !scales_dev || !data_t_dev != !scales_t_dev || (!data_dev && !data_t_dev)) return CONV2D_ERR_INVALID;
    if (rows > mx::MAX_EXTENT || cols > mx::MAX_EXTENT) return CONV2D_ERR_UNSUPPORTED;
    if (rows == 0) return CONV2D_OK;
    if (!x_dev) return CONV2D_ERR_INVALID;
    for (const void* p : {static_cast<const void*>(data_dev), static_cast<const void*>(scales_dev),
                          static_cast<const void*>(data_t_dev), static_cast<const void*>(scales_t_dev)})
        if (reinterpret_cast<uintptr_t>(p) % 16) return CONV2D_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(x_dev) % (x_dtype == CONV2D_OUT_BF16 ? 2 : 4)) return CONV2D_ERR_ALIGNMENT;
    mx::QuantParams k{};
    k.rows = rows;
    k.cols = cols;
    k.x_stride = x_stride;
    k.row_tiles = mx::cdiv<int64_t>(rows, mx::Q_TILE);
    k.col_tiles = mx::cdiv<int64_t>(cols, mx::Q_TILE);
    k.data = static_cast<uint8_t*>(data_dev);
    k.scales = static_cast<uint8_t*>(scales_dev);
    k.data_t = static_cast<uint8_t*>(data_t_dev);
    k.scales_t = static_cast<uint8_t*>(scales_t_dev);
    const int64_t grid = k.row_tiles * k.col_tiles;
    if (grid > mx::MAX_EXTENT) return CONV2D_ERR_UNSUPPORTED;
    if (x_dtype == CONV2D_OUT_BF16)
        mx::quantize_kernel<<<static_cast<unsigned>(grid), mx::Q_THREADS, 0, stream>>>(static_cast<const __nv_bfloat16*>(x_dev), k);
    else
        mx::quantize_kernel<<<static_cast<unsigned>(grid), mx::Q_THREADS, 0, stream>>>(static_cast<const float*>(x_dev), k);
    return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

extern "C" int mxfp4_dequantize(int64_t rows, int64_t cols, const void* data_dev, const void* scales_dev, void* y_dev,
                                int32_t y_dtype, conv2d_stream_t stream)
{
    if (rows < 0 || cols < 1 || (y_dtype != CONV2D_OUT_F32 && y_dtype != CONV2D_OUT_BF16)) return CONV2D_ERR_INVALID;
    if (rows > mx::MAX_EXTENT || cols > mx::MAX_EXTENT) return CONV2D_ERR_UNSUPPORTED;
    if (rows == 0) return CONV2D_OK;
    if (!data_dev || !scales_dev || !y_dev) return CONV2D_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(data_dev) % 16 || reinterpret_cast<uintptr_t>(scales_dev) % 16 ||
        reinterpret_cast<uintptr_t>(y_dev) % 16)
        return CONV2D_ERR_ALIGNMENT;
    const int64_t n = rows * mx::cdiv<int64_t>(cols, mx::BLOCK) * 4;
    const unsigned grid = static_cast<unsigned>(mx::cdiv<int64_t>(n, 256) < 152 * 64 ? mx::cdiv<int64_t>(n, 256) : 152 * 64);
    const uint8_t *d = static_cast<const uint8_t*>(data_dev), *s = static_cast<const uint8_t*>(scales_dev);
    if (y_dtype == CONV2D_OUT_BF16)
        mx::dequantize_kernel<<<grid, 256, 0, stream>>>(d, s, static_cast<__nv_bfloat16*>(y_dev), rows, cols);
    else
        mx::dequantize_kernel<<<grid, 256, 0, stream>>>(d, s, static_cast<float*>(y_dev), rows, cols);
    return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}
