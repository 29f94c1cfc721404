// Kernel parameters of the layer normalisation kernels.
#pragma once

#include "mx_common.cuh"

namespace sgb {
namespace ln {

struct FwdParams {
    const void* x;
    void* y;
    int64_t rows, x_stride, y_stride, padded_rows;
    int cols;
    float eps, inv_cols;
    const float *weight, *bias;
    float *mean, *rstd;
    uint8_t *data, *scales;
};

struct BwdParams {
    const void *x, *dy;
    void* dx;
    int64_t rows, x_stride, dy_stride, chunk;
    int cols;
    float inv_cols;
    const float *mean, *rstd, *weight;
    float *dweight, *dbias, *part;  // part: [chunks][2][cols]
    int chunks;
};

// A row of `cols` elements is shared by `threads` threads of `elems` elements each; threads = 0: it is too wide
// for a block's registers.  128 threads and more are a block of their own; fewer share a block of 256.
struct RowShape {
    int threads, elems;
};

// The narrowest shape that holds the row: groups inside a warp up to 512 columns (no barriers), then blocks
// of 8 and of 16 elements to a thread.
__host__ __device__ constexpr RowShape row_shape(int64_t cols)
{
    return cols <= 64 ? RowShape{8, 8} : cols <= 128 ? RowShape{16, 8} : cols <= 256 ? RowShape{32, 8} : cols <= 512 ? RowShape{32, 16}
         : cols <= 1024 ? RowShape{128, 8} : cols <= 2048 ? RowShape{256, 8} : cols <= 4096 ? RowShape{256, 16}
         : cols <= 8192 ? RowShape{512, 16} : cols <= 16384 ? RowShape{1024, 16} : RowShape{0, 0};
}

__host__ __device__ constexpr int block_threads(int threads) { return threads <= 32 ? 256 : threads; }
__host__ __device__ constexpr int rows_per_block(RowShape s) { return block_threads(s.threads) / s.threads; }

// Blocks that stay on an SM, by the registers their rows, weights and sums need: forward 64 a thread for 8
// elements and 80 for 16; backward 85 (a row's 8 elements), 128 for 16.
__host__ __device__ constexpr int fwd_resident(RowShape s)
{
    const int t = block_threads(s.threads);
    return s.elems == 8 ? 1024 / t : t >= 512 ? 1 : 768 / t;
}
__host__ __device__ constexpr int bwd_resident(RowShape s)
{
    const int t = block_threads(s.threads);
    return s.elems == 8 && t <= 256 ? 640 / t : t >= 512 ? 1 : 512 / t;
}

constexpr int SMS = mx::SMS;

// Launches by element types (one translation unit each); `vec`: rows can be read and written in vectors.
// False: the row does not fit and nothing was launched.
template <typename TX, typename TY>
bool launch_fwd_rows(const FwdParams& p, bool vec, cudaStream_t stream);
template <typename TX, typename TY>
bool launch_bwd_rows(const BwdParams& p, bool vec, int grid, cudaStream_t stream);

}  // namespace ln
}  // namespace sgb
