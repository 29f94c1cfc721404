// Kernel parameters of the layer normalisation kernels.
#pragma once

#include <atomic>

#include "mx_common.cuh"

namespace sgb {
namespace ln {

struct FwdParams {
    const void* x;
    void* y;
    int64_t rows, x_stride, y_stride, padded_rows;
    int cols, span;  // span: columns that a group has to hold, with what may stand in front of an unaligned row
    float eps, inv_cols;
    const float *weight, *bias;
    float *mean, *rstd;
    uint8_t *data, *scales;
};

struct BwdParams {
    const void *x, *dy;
    void* dx;
    int64_t rows, x_stride, dy_stride, chunk;
    int cols, span;
    float inv_cols;
    const float *mean, *rstd, *weight;
    float *dweight, *dbias, *part;  // part: [chunks][2][cols]
    int chunks;
};

// A row is shared by `threads` threads of `elems` elements each.  Up to 32 threads are a group inside a warp, and a
// block of 256 has 256/threads rows; more are a block of their own, of at most `most` threads (by which its kernel
// is compiled).  threads = 0: the row is too wide for a block's registers.
struct RowShape {
    int threads, elems, most;
};

// The fewest threads that hold the row: groups inside a warp up to 512 columns (no barriers), then blocks of whole
// warps of 8, 16 and 32 elements to a thread.
__host__ __device__ constexpr RowShape row_shape(int64_t cols)
{
    const int n = static_cast<int>(cols);
    return cols <= 64 ? RowShape{8, 8, 256} : cols <= 128 ? RowShape{16, 8, 256} : cols <= 256 ? RowShape{32, 8, 256}
         : cols <= 512 ? RowShape{32, 16, 256} : cols <= 2048 ? RowShape{(n + 255) / 256 * 32, 8, 256}
         : cols <= 4096 ? RowShape{(n + 511) / 512 * 32, 16, 256} : cols <= 8192 ? RowShape{(n + 511) / 512 * 32, 16, 512}
         : cols <= 16384 ? RowShape{(n + 1023) / 1024 * 32, 32, 512} : RowShape{0, 0, 0};
}

__host__ __device__ constexpr int block_threads(RowShape s) { return s.threads <= 32 ? s.most : s.threads; }
__host__ __device__ constexpr int rows_per_block(RowShape s) { return s.threads <= 32 ? s.most / s.threads : 1; }

// Threads that stay on an SM, by the registers that rows, weights and sums need: forward 64 to a thread for 8
// elements, 85 for 16, 128 for 16 or 32 in wide blocks; backward 85 and 128.  And the blocks of a shape that they make.
__host__ __device__ constexpr int fwd_threads(RowShape s) { return s.most == 512 ? 512 : s.elems == 8 ? 1024 : 768; }
__host__ __device__ constexpr int bwd_threads(RowShape s) { return s.most == 512 || s.elems > 8 ? 512 : 768; }
__host__ __device__ constexpr int fwd_resident(RowShape s) { return fwd_threads(s) / block_threads(s); }
__host__ __device__ constexpr int bwd_resident(RowShape s) { return bwd_threads(s) / block_threads(s); }

// Rows of a block's ring: up to four, within 200 KB of an SM's shared memory.
__host__ __device__ constexpr int ring_depth(RowShape s, int x_bytes, int y_bytes)
{
    const int n = 200 * 1024 / ((y_bytes ? bwd_threads(s) : fwd_threads(s)) * s.elems * (x_bytes + y_bytes));
    return n > 4 ? 4 : n;
}

constexpr int SMS = mx::SMS;

// Blocks for `rows` rows: the resident ones at most, and for a row to a block a multiple of 8, so that a block's rows
// start at the same place within 16 bytes.
__host__ __device__ constexpr int64_t row_blocks(int64_t rows, RowShape s, int resident)
{
    const int per = rows_per_block(s);
    const int64_t n = per == 1 ? mx::cdiv<int64_t>(rows, 8) * 8 : mx::cdiv<int64_t>(rows, per);
    return n < SMS * resident ? n : SMS * resident;
}

// Lets a kernel have `bytes` of dynamic shared memory; asked of the driver once per device.
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done)
{
    if (bytes <= 48 * 1024) return true;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev < 64) done.fetch_or(bit, std::memory_order_release);
    return true;
}

// Launches by element types (one translation unit each); `vec`: rows can be read and written in vectors.
// CONV2D_ERR_UNSUPPORTED: the row does not fit and nothing was launched.
template <typename TX, typename TY>
int launch_fwd_rows(const FwdParams& p, bool vec, cudaStream_t stream);
template <typename TX, typename TY>
int launch_bwd_rows(const BwdParams& p, bool vec, int grid, cudaStream_t stream);

}  // namespace ln
}  // namespace sgb
