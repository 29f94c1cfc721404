// Microscaled 4-bit matrices: quantisation by rows, by columns or both, and the way back.
#include "mxfp4.h"

#include "mx_common.cuh"
#include "ptx.cuh"

namespace sgb {
namespace mx {

constexpr int64_t MAX_EXTENT = (int64_t(1) << 31) - 1;

bool extents_ok(int64_t rows, int64_t cols) { return rows >= 1 && cols >= 1 && rows <= MAX_EXTENT && cols <= MAX_EXTENT; }

struct QuantParams {
    int64_t rows, cols, x_stride;
    int64_t row_tiles, col_tiles;  // of 128 x 128 elements
    uint8_t *data, *scales, *data_t, *scales_t;
};

// A block of threads takes a tile of 128 x 128 elements, which is one scale tile of either form, through shared memory, so
// that both forms come from one reading of x.  A thread quantises 8 neighbouring elements of a row (4 or 8 of them make
// a block's 32), or 32 elements of one column (two columns where x is bf16, which come as one word); what it makes is
// gathered in shared memory and leaves in whole rows: 64 bytes of data, 512 bytes of scales.  x is read once and 17/32 of a byte
// written for each element of each form; bound by issue, some 17 instructions an element for both forms (16384 x 4096 bf16: rows
// 38 us, columns 34, both 50, 4.1 TB/s; fp32: rows 67, columns 61, both 79, 4.3 TB/s).
constexpr int Q_TILE = 128;
constexpr int Q_THREADS = 256;

template <typename T>
struct alignas(16) QuantTile {
    T x[Q_TILE][Q_TILE];
    uint8_t out[Q_TILE * Q_TILE / 2];  // [row or column][64 bytes], see out_at
    uint8_t scales[TILE_BYTES];
};

// Where block q of line l is gathered: lines by twos in 128 bytes, whose eight 16-byte units are permuted by the
// line so that threads with lines in turn write to different banks.
__device__ __forceinline__ int out_at(int l, int q) { return (l >> 1) * 128 + ((((l & 1) * 4 + q) ^ ((l >> 1) & 7)) << 4); }

// The larger absolute value, as bits; bf16 values come in pairs and are compared as pairs.  A NaN stays (its bits
// are above every number's).
__device__ __forceinline__ uint32_t join_max(uint32_t m, uint32_t v, float) { return max(m, v & 0x7fffffffu); }
__device__ __forceinline__ uint32_t join_max(uint32_t m, uint32_t v, __nv_bfloat16)
{
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(const T* __restrict__ x, const QuantParams p)
{
    extern __shared__ uint8_t raw[];
    QuantTile<T>& s = *reinterpret_cast<QuantTile<T>*>(raw);
    const int64_t rb = blockIdx.x / p.col_tiles, cb = blockIdx.x - rb * p.col_tiles;
    const int64_t r0 = rb * Q_TILE, c0 = cb * Q_TILE;
    const int rows = static_cast<int>(p.rows - r0 < Q_TILE ? p.rows - r0 : Q_TILE);
    const int cols = static_cast<int>(p.cols - c0 < Q_TILE ? p.cols - c0 : Q_TILE);
    const T* src = x + r0 * p.x_stride + c0;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T), PER = Q_TILE / V, STEP = Q_THREADS / PER;
        const int c = threadIdx.x % PER * V;
        uint4 v[Q_TILE / STEP];
#pragma unroll
        for (int i = 0; i < Q_TILE / STEP; ++i) {
            const int r = threadIdx.x / PER + i * STEP;
            v[i] = r < rows && c < cols ? __ldg(reinterpret_cast<const uint4*>(src + r * p.x_stride + c)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < Q_TILE / STEP; ++i) *reinterpret_cast<uint4*>(&s.x[threadIdx.x / PER + i * STEP][c]) = v[i];
    } else {
        const int c = threadIdx.x % Q_TILE;
#pragma unroll 16
        for (int r = threadIdx.x / Q_TILE; r < Q_TILE; r += Q_THREADS / Q_TILE)
            s.x[r][c] = r < rows && c < cols ? src[r * p.x_stride + c] : T(0.f);
    }
    __syncthreads();

    const int64_t row_blocks = cdiv<int64_t>(p.rows, BLOCK), col_blocks = cdiv<int64_t>(p.cols, BLOCK);
    // Copies the gathered lines of `n` rows (of the form's matrix) and the scale tile; `left` blocks of a line exist.
    auto flush = [&](uint8_t* data, uint8_t* scales, int64_t line0, int n, int64_t pitch, int64_t block0, int64_t left, int64_t tile) {
        __syncthreads();
        const int q = threadIdx.x % TILE_BLOCKS;
        for (int l = threadIdx.x / TILE_BLOCKS; l < n; l += Q_THREADS / TILE_BLOCKS)
            if (q < left)
                *reinterpret_cast<uint4*>(data + ((line0 + l) * pitch + block0 + q) * 16) =
                    *reinterpret_cast<const uint4*>(s.out + out_at(l, q));
        if (threadIdx.x < TILE_BYTES / 16)
            reinterpret_cast<uint4*>(scales + tile * TILE_BYTES)[threadIdx.x] = reinterpret_cast<const uint4*>(s.scales)[threadIdx.x];
    };

    if (p.data) {
        const int lane = threadIdx.x % 16, c = 8 * lane;
#pragma unroll
        for (int i = 0; i < Q_TILE / 16; ++i) {
            const int r = threadIdx.x / 16 + 16 * i;
            float v[8];
            uint32_t m = 0;
            if constexpr (sizeof(T) == 2) {
                const uint4 w = *reinterpret_cast<const uint4*>(&s.x[r][c]);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m = join_max(m, u[j], T());
                    v[2 * j] = __uint_as_float(u[j] << 16);
                    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
                }
                m = max(m << 16, m & 0xffff0000u);
            } else {
                float largest = 0.f;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    v[j] = s.x[r][c + j];
                    v[j + 1] = s.x[r][c + j + 1];
                    largest = max_abs3(largest, v[j], v[j + 1]);
                }
                m = __float_as_uint(largest);
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t byte = scale_byte(m);
            const float inv = inverse_scale(byte);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 w = mul2(make_float2(v[j], v[j + 1]), make_float2(inv, inv));
                v[j] = w.x;
                v[j + 1] = w.y;
            }
            *reinterpret_cast<uint32_t*>(s.out + out_at(r, lane / 4) + 4 * (lane % 4)) = pack_e2m1x8(v);
            if (lane % 4 == 0) s.scales[(r % 32) * 16 + r / 32 * 4 + lane / 4] = static_cast<uint8_t>(byte);
        }
        flush(p.data, p.scales, r0, rows, col_blocks, cb * TILE_BLOCKS, col_blocks - cb * TILE_BLOCKS, rb * p.col_tiles + cb);
        __syncthreads();
    }
    if (p.data_t) {
        constexpr int PAIR = 4 / sizeof(T);  // columns in a word
        constexpr int WORDS = Q_TILE / PAIR;
        for (int u = threadIdx.x; u < WORDS * TILE_BLOCKS; u += Q_THREADS) {
            const int w = u % WORDS, g = u / WORDS;
            uint32_t v[BLOCK], m = 0;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                v[i] = reinterpret_cast<const uint32_t*>(&s.x[g * BLOCK + i][0])[w];
                m = join_max(m, v[i], T());
            }
#pragma unroll
            for (int h = 0; h < PAIR; ++h) {
                const int c = w * PAIR + h;
                const uint32_t byte = scale_byte(PAIR == 1 ? m : h ? m & 0xffff0000u : m << 16);
                const float inv = inverse_scale(byte);
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const uint32_t b0 = v[8 * q + j], b1 = v[8 * q + j + 1];
                        const float2 w = mul2(make_float2(__uint_as_float(PAIR == 1 ? b0 : h ? b0 & 0xffff0000u : b0 << 16),
                                                          __uint_as_float(PAIR == 1 ? b1 : h ? b1 & 0xffff0000u : b1 << 16)),
                                              make_float2(inv, inv));
                        f[j] = w.x;
                        f[j + 1] = w.y;
                    }
                    o[q] = pack_e2m1x8(f);
                }
                *reinterpret_cast<uint4*>(s.out + out_at(c, g)) = make_uint4(o[0], o[1], o[2], o[3]);
                s.scales[(c % 32) * 16 + c / 32 * 4 + g] = static_cast<uint8_t>(byte);
            }
        }
        flush(p.data_t, p.scales_t, c0, cols, row_blocks, rb * TILE_BLOCKS, row_blocks - rb * TILE_BLOCKS, cb * p.row_tiles + rb);
    }
}

// A thread takes 8 elements: 4 bytes in, 16 or 32 out (in one or two 16-byte stores where rows are whole vectors; else a
// warp's 256 elements go through shared memory and leave element by element in order).
// Bound by HBM once four rows' loads are in flight: 16384 x 4096 to bf16 31 us, 5.5 TB/s (one row at a time 34), to fp32 51 us, 6.0 TB/s (57).
// Other widths are bound by their way through shared memory: 16384 x 4093 79 us to bf16 and 78 to fp32; 4097 columns, whose third block
// of 256 threads across has 4 at work, 123 and 121.
constexpr int D_THREADS = 256;

template <typename T, bool VEC>
__global__ void __launch_bounds__(D_THREADS) dequantize_kernel(const uint8_t* __restrict__ data, const uint8_t* __restrict__ scales, T* y,
                                                               int64_t rows, int64_t cols, int lanes_log2)
{
    // a thread keeps its 8 columns, 1 << lanes_log2 threads side by side, and goes down the rows
    __shared__ float gather[VEC ? 1 : D_THREADS][9];
    const int64_t blocks = cdiv<int64_t>(cols, BLOCK), btiles = cdiv<int64_t>(blocks, TILE_BLOCKS);
    const int64_t words = blocks * 4;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1));
    constexpr int DEPTH = 4;  // neighbouring rows, on their way at once
    const int64_t per = (D_THREADS >> lanes_log2) * DEPTH, step = gridDim.y * per;
    const int64_t r0 = blockIdx.y * per + (threadIdx.x >> lanes_log2) * DEPTH;
    const int64_t lead = blockIdx.y * per + ((threadIdx.x & ~31) >> lanes_log2) * DEPTH;  // of the warp, whose lanes stay together
    const uint8_t* scale_col = scales + (w >> 4) * TILE_BYTES + ((w >> 2) & 3);
    const int lane = threadIdx.x & 31;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    for (int64_t k0 = 0; lead + k0 < rows; k0 += step) {
        uint32_t words_of[DEPTH] = {}, scale_of[DEPTH] = {};
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int64_t r = r0 + k0 + d;
            if (r < rows && w < words) {
                words_of[d] = __ldg(reinterpret_cast<const uint32_t*>(data) + r * words + w);
                scale_of[d] = __ldg(scale_col + scale_at(r, 0, btiles));
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int64_t r = r0 + k0 + d;
            float2 v[4];
            unpack_e2m1x8(v, words_of[d]);
            const float s = scale_value(scale_of[d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], make_float2(s, s));
            if constexpr (VEC) {
                if (r < rows && w * 8 < cols) {
                    T* out = y + r * cols + w * 8;
                    if constexpr (sizeof(T) == 4) {
                        if (reinterpret_cast<uintptr_t>(out) % 32 == 0) {  // a whole sector to a thread
                            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(v[0].x), "f"(v[0].y),
                                         "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
                                         : "memory");
                        } else {
                            reinterpret_cast<float4*>(out)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
                            reinterpret_cast<float4*>(out)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
                        }
                    } else {
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x, v[j].y);
                            o[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            } else {
                float(*mine)[9] = gather + (threadIdx.x & ~31);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mine[lane][2 * j] = v[j].x;
                    mine[lane][2 * j + 1] = v[j].y;
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int from = 4 * e + lane / 8;  // the thread whose element this is
                    const int64_t fr = __shfl_sync(0xffffffffu, r, from), fw = __shfl_sync(0xffffffffu, w, from);
                    const int64_t c = fw * 8 + lane % 8;
                    if (fr < rows && c < cols) from_float(y[fr * cols + c], mine[from][lane % 8]);
                }
            }
        }
    }
}

// One block to a tile.
template <typename T, bool VEC>
int launch_quantize(const T* x, const QuantParams& p, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    constexpr int smem = sizeof(QuantTile<T>);
    if (!allow_smem(quantize_kernel<T, VEC>, smem, done)) return CONV2D_ERR_CUDA;
    return launch(quantize_kernel<T, VEC>, p.row_tiles * p.col_tiles, Q_THREADS, smem, stream, 1, x, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

template <typename T>
int quantize(const void* x, const QuantParams& p, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool vec = p.cols % V == 0 && p.x_stride % V == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    return vec ? launch_quantize<T, true>(static_cast<const T*>(x), p, stream) : launch_quantize<T, false>(static_cast<const T*>(x), p, stream);
}

template <typename T>
int dequantize(const uint8_t* data, const uint8_t* scales, void* y, int64_t rows, int64_t cols, cudaStream_t stream)
{
    const int64_t words = cdiv<int64_t>(cols, BLOCK) * 4;
    int lanes_log2 = 2;
    while (lanes_log2 < 8 && (int64_t(1) << lanes_log2) < words) ++lanes_log2;
    // Eight blocks to an SM at most: they stay, and go down the rows.
    const int64_t across = cdiv<int64_t>(words, int64_t(1) << lanes_log2), down = cdiv<int64_t>(rows, (D_THREADS >> lanes_log2) * 4);
    const int64_t most = cdiv<int64_t>(SMS * 8, across) < 65535 ? cdiv<int64_t>(SMS * 8, across) : 65535;
    if (across > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(down < most ? down : most));
    const auto kernel = cols % 8 == 0 ? dequantize_kernel<T, true> : dequantize_kernel<T, false>;
    return launch(kernel, grid, D_THREADS, 0, stream, 1, data, scales, static_cast<T*>(y), rows, cols, lanes_log2) == cudaSuccess ? CONV2D_OK
                                                                                                                                : CONV2D_ERR_CUDA;
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
    return x_dtype == CONV2D_OUT_BF16 ? mx::quantize<__nv_bfloat16>(x_dev, k, stream) : mx::quantize<float>(x_dev, k, stream);
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
    const uint8_t *d = static_cast<const uint8_t*>(data_dev), *s = static_cast<const uint8_t*>(scales_dev);
    return y_dtype == CONV2D_OUT_BF16 ? mx::dequantize<__nv_bfloat16>(d, s, y_dev, rows, cols, stream)
                                      : mx::dequantize<float>(d, s, y_dev, rows, cols, stream);
}
