// Kernel parameters of the layer normalisation kernels.
#pragma once

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
    int64_t rows, x_stride, dy_stride;
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

// A row's two sums cost each of its threads some 40 instructions of shuffles whatever it holds, so threads hold much
// where there are rows enough to keep the SMs busy with few threads to a row, and 16-bit rows, which bring twice the
// elements for their bytes, hold twice what fp32 rows do.  (bf16, 65536 x 1024 forward: 32 elements 45 us, 8 elements 54;
// fp32, 401408 x 64 backward: 16 elements 69 us, 8 elements 57.)
__host__ __device__ constexpr bool many_rows(int64_t rows, int x_bytes, int threads) { return x_bytes == 2 && rows * threads >= 4 * 512 * 152; }

// The shape of `elems` elements to a thread in whole warps; 0 threads where that is over `most`.
__host__ __device__ constexpr RowShape warps_of(int n, int elems, int most)
{
    const int t = (n + 32 * elems - 1) / (32 * elems) * 32;
    return t <= most ? RowShape{t, elems, most} : RowShape{0, 0, 0};
}

// Up to 512 columns: groups inside a warp.
__host__ __device__ constexpr RowShape group_shape(int n, bool many)
{
    return n > 256 ? RowShape{32, 16, 256} : many ? (n <= 64 ? RowShape{4, 16, 256} : n <= 128 ? RowShape{8, 16, 256} : RowShape{16, 16, 256})
                                                  : (n <= 64 ? RowShape{8, 8, 256} : n <= 128 ? RowShape{16, 8, 256} : RowShape{32, 8, 256});
}

// Forward: a warp to a row of up to 1024 columns where there are many rows and those nearly fill it, else blocks of 8, 16 or 32
// elements to a thread.  `whole`: rows are whole vectors (others need registers for masks; of 4097 to 6144
// columns two blocks of at most 384 threads stay on an SM instead of one: 16380 x 4097, forward bf16 65 us against 97, fp32 89 against
// 113, quantised bf16 95 against 125).
__host__ __device__ constexpr RowShape fwd_shape(int64_t rows, int64_t cols, int x_bytes, bool whole)
{
    if (cols > 16384) return RowShape{0, 0, 0};
    const int n = static_cast<int>(cols);
    if (n <= 512) return group_shape(n, many_rows(rows, x_bytes, 16));
    if (n > 768 && n <= 1024 && whole && many_rows(rows, x_bytes, 32)) return RowShape{32, 32, 256};
    return n <= (many_rows(rows, x_bytes, 64) ? 1024 : 2048) ? warps_of(n, 8, 256) : n <= 4096 ? warps_of(n, 16, 256)
         : n <= 8192 && !whole                               ? warps_of(n, 16, n <= 6144 ? 384 : 512) : warps_of(n, 32, 512);
}

// Backward: the sums of dweight and dbias leave registers for 16 elements; above 8192 columns dx alone takes 32.
__host__ __device__ constexpr RowShape bwd_shape(int64_t rows, int64_t cols, int x_bytes, bool whole)
{
    if (cols > 16384) return RowShape{0, 0, 0};
    const int n = static_cast<int>(cols);
    if (n <= 512) return group_shape(n, many_rows(rows, x_bytes, 16));
    if (n > 8192) return warps_of(n, 32, 512);
    const bool wide = n > 2048 || (many_rows(rows, x_bytes, 64) && whole && (n + 511) / 512 * 512 <= n + n / 4);
    return wide ? warps_of(n, 16, n <= 4096 ? 256 : 512) : warps_of(n, 8, 256);
}

__host__ __device__ constexpr int block_threads(RowShape s) { return s.threads <= 32 ? s.most : s.threads; }
__host__ __device__ constexpr int rows_per_block(RowShape s) { return s.threads <= 32 ? s.most / s.threads : 1; }

// Threads that stay on an SM, by the registers that rows, weights and sums need: forward 64 to a thread of 8 elements, 85 of
// 16 in blocks of at most 384 threads, else 128; backward 85 and 128.  And the blocks of a shape that they make.
__host__ __device__ constexpr int fwd_threads(RowShape s) { return s.elems == 8 ? 1024 : s.elems == 16 && s.most <= 384 ? 768 : 512; }
__host__ __device__ constexpr int bwd_threads(RowShape s) { return s.elems == 8 ? 768 : 512; }
__host__ __device__ constexpr int fwd_resident(RowShape s) { return fwd_threads(s) / block_threads(s); }
__host__ __device__ constexpr int bwd_resident(RowShape s) { return bwd_threads(s) / block_threads(s); }

// Rows of a block's ring: some 72 KB of them on an SM, as more in flight slows HBM down (bf16, 32768 x 4096 forward, rows of all
// blocks 24 KB: two 89.5 us, three 88.4, four 93.3; backward, 32 KB: two to five 141 to 142), but two at least where they fit.
__host__ __device__ constexpr int ring_depth(RowShape s, int x_bytes, int y_bytes)
{
    const int row = (y_bytes ? bwd_threads(s) : fwd_threads(s)) * s.elems * (x_bytes + y_bytes);
    const int n = 72 * 1024 / row;
    return n > 4 ? 4 : n >= 2 ? n : 2 * row <= 200 * 1024 ? 2 : 1;
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

// Backward: each block also writes a part of the sums over the rows, as many bytes as two rows of them; so blocks take four rows
// at least where that leaves one to an SM.
__host__ __device__ constexpr int64_t bwd_blocks(int64_t rows, RowShape s)
{
    const int64_t n = row_blocks(rows, s, bwd_resident(s));
    const int64_t fourth = mx::cdiv<int64_t>(rows, int64_t(32) * rows_per_block(s)) * 8, few = fourth > SMS ? fourth : SMS;
    return n < few ? n : few;
}

// Launches by element types (one translation unit each); `vec`: rows can be read and written in vectors.
// CONV2D_ERR_UNSUPPORTED: the row does not fit and nothing was launched.
template <typename TX, typename TY>
int launch_fwd_rows(const FwdParams& p, bool vec, cudaStream_t stream);
template <typename TX, typename TY>
int launch_bwd_rows(const BwdParams& p, bool vec, int grid, cudaStream_t stream);

}  // namespace ln
}  // namespace sgb
