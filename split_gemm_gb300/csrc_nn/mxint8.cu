// Activation checkpoints in 8 bits: quantisation and the way back.
#include "mxint8.h"

#include <type_traits>

#include "mxint8.cuh"

namespace sgb {
namespace mx {

constexpr int64_t INT8_MOST = (int64_t(1) << 31) - 32;

bool int8_extents_ok(int64_t rows, int64_t cols) { return rows >= 1 && cols >= 1 && rows <= INT8_MOST && cols <= INT8_MOST; }

constexpr int I_THREADS = 256;
constexpr int I_DEPTH = 4;  // neighbouring rows, on their way at once

// The elements that a thread takes side by side: 32 bytes of x.
template <typename T>
constexpr int SPAN = 32 / sizeof(T);

// A thread keeps its columns, 1 << lanes_log2 threads side by side, and goes down the rows; 2 (bf16) or 4 (fp32) threads hold a block and
// find its largest value by shuffles.  x is read once and 33/32 bytes are written for each element: HBM binds.
// 32768 x 4096 bf16: 62 us, 6.5 TB/s.
template <typename T, bool VEC>
__global__ void __launch_bounds__(I_THREADS) quantize_int8(const T* __restrict__ x, uint8_t* __restrict__ data, uint8_t* __restrict__ scales,
                                                           int64_t rows, int64_t cols, int64_t x_stride, int lanes_log2)
{
    constexpr int E = SPAN<T>, LANES = BLOCK / E;
    const int64_t blocks = cdiv<int64_t>(cols, BLOCK);
    const int64_t w = (static_cast<int64_t>(blockIdx.x) << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1));
    const int64_t c = w * E;
    const bool inside = c < blocks * BLOCK;
    const int valid = static_cast<int>(c >= cols ? 0 : cols - c < E ? cols - c : E);
    const int64_t per = (I_THREADS >> lanes_log2) * I_DEPTH, step = gridDim.y * per;
    const int64_t r0 = blockIdx.y * per + (threadIdx.x >> lanes_log2) * I_DEPTH;
    const int64_t lead = blockIdx.y * per + ((threadIdx.x & ~31) >> lanes_log2) * I_DEPTH;  // of the warp, whose lanes stay together
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    for (int64_t k0 = 0; lead + k0 < rows; k0 += step) {
        uint32_t u[I_DEPTH][8];
#pragma unroll
        for (int d = 0; d < I_DEPTH; ++d) {
            const int64_t r = r0 + k0 + d;
            const bool live = r < rows && valid > 0;
            if constexpr (VEC) {
                const uint4* src = reinterpret_cast<const uint4*>(x + (live ? r * x_stride + c : 0));
                const uint4 z = make_uint4(0, 0, 0, 0);
                const uint4 a = live ? __ldg(src) : z, b = live && valid > E / 2 ? __ldg(src + 1) : z;
                u[d][0] = a.x, u[d][1] = a.y, u[d][2] = a.z, u[d][3] = a.w;
                u[d][4] = b.x, u[d][5] = b.y, u[d][6] = b.z, u[d][7] = b.w;
            } else {
                load_any<8, sizeof(T)>(u[d], x + (live ? r * x_stride + c : 0), live ? valid * static_cast<int>(sizeof(T)) : 0);
            }
        }
#pragma unroll
        for (int d = 0; d < I_DEPTH; ++d) {
            const int64_t r = r0 + k0 + d;
            float v[E];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[2 * i] = __uint_as_float(u[d][i] << 16);
                    v[2 * i + 1] = __uint_as_float(u[d][i] & 0xffff0000u);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[d][i]);
            }
            float largest = fabsf(v[0]);
#pragma unroll
            for (int i = 0; i < E; i += 2) largest = max_abs3(largest, v[i], v[i + 1]);
            uint32_t m = abs_bits(largest);
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t byte = int8_scale_byte(m);
            const float inv = int8_inverse(byte);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 s = mul2(make_float2(v[i], v[i + 1]), make_float2(inv, inv));
                v[i] = s.x;
                v[i + 1] = s.y;
            }
            uint32_t o[E / 4];
#pragma unroll
            for (int i = 0; i < E / 4; ++i) o[i] = byte == 255u ? 0u : pack_int8x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (r < rows && inside) {
                uint8_t* dst = data + r * (blocks * BLOCK) + c;
                if constexpr (E == 16)
                    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                else
                    *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
                if (w % LANES == 0) scales[r * blocks + w / LANES] = static_cast<uint8_t>(byte);
            }
        }
    }
}

// Stores E values from element address `out` on, those below `valid`; VEC: `out` is a whole vector's.
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* out, const float2 (&v)[E / 2])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) reinterpret_cast<float4*>(out)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    } else {
        uint32_t o[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
            o[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int i = 0; i < E / 8; ++i) reinterpret_cast<uint4*>(out)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
}

// A thread makes 32 aligned bytes of y; HBM binds.  32768 x 4096 to bf16: 71 us, 5.8 TB/s.  Rows of y that do not begin at 16 bytes (VEC = false): `off` elements of the row before stand in
// front of a row's first vector, so a thread's elements lie `off` to the left in data, which is read from any byte, and in one or two
// blocks; the first and last vector of a row are stored by elements.
template <typename T, bool VEC>
__global__ void __launch_bounds__(I_THREADS) dequantize_int8(const uint8_t* __restrict__ data, const uint8_t* __restrict__ scales, T* __restrict__ y,
                                                             int64_t rows, int64_t cols, int lanes_log2)
{
    constexpr int E = SPAN<T>, LANES = BLOCK / E, V = 16 / sizeof(T);
    const int64_t blocks = cdiv<int64_t>(cols, BLOCK);
    const int64_t w = (static_cast<int64_t>(blockIdx.x) << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1));
    const int64_t per = (I_THREADS >> lanes_log2) * I_DEPTH, step = gridDim.y * per;
    const int64_t r0 = blockIdx.y * per + (threadIdx.x >> lanes_log2) * I_DEPTH;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (VEC && w * E >= cols) return;
    for (int64_t k0 = 0; r0 + k0 < rows; k0 += step) {
        if constexpr (VEC) {
            uint32_t u[I_DEPTH][E / 4], s[I_DEPTH];
#pragma unroll
            for (int d = 0; d < I_DEPTH; ++d) {
                const int64_t r = r0 + k0 + d < rows ? r0 + k0 + d : r0 + k0;
                const uint8_t* src = data + r * (blocks * BLOCK) + w * E;
                if constexpr (E == 16) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4*>(src));
                    u[d][0] = q.x, u[d][1] = q.y, u[d][2] = q.z, u[d][3] = q.w;
                } else {
                    const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
                    u[d][0] = q.x, u[d][1] = q.y;
                }
                s[d] = __ldg(scales + r * blocks + w / LANES);
            }
#pragma unroll
            for (int d = 0; d < I_DEPTH; ++d) {
                const int64_t r = r0 + k0 + d;
                float2 v[E / 2];
                const float f = scale_value(s[d]);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    float2 q[2];
                    unpack_int8x4(q, u[d][i]);
                    v[2 * i] = mul2(q[0], make_float2(f, f));
                    v[2 * i + 1] = mul2(q[1], make_float2(f, f));
                }
                if (r < rows) {
                    T* out = y + r * cols + w * E;
                    if (w * E + E <= cols) {
                        store_vec<T, E>(out, v);
                    } else {  // a whole number of 16-byte vectors is left
#pragma unroll
                        for (int i = 0; i < E / V; ++i) {
                            float2 h[V / 2];
#pragma unroll
                            for (int j = 0; j < V / 2; ++j) h[j] = v[i * V / 2 + j];
                            if (w * E + i * V < cols) store_vec<T, V>(out + i * V, h);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int d = 0; d < I_DEPTH; ++d) {
                const int64_t r = r0 + k0 + d;
                if (r >= rows) break;
                T* row = y + r * cols;
                const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
                const int64_t c = w * E - off;  // of the first element; below 0 in a row's first vector
                if (c >= cols) continue;
                const int skip = c < 0 ? static_cast<int>(-c) : 0;  // elements in front of the row
                const int64_t first = c + skip;
                const int64_t have = blocks * BLOCK - first;
                uint32_t u[4];
                load_any<4, 1>(u, data + r * (blocks * BLOCK) + first, static_cast<int>(have < 16 ? have : 16));
                const int64_t b = first / BLOCK;
                const float f0 = scale_value(__ldg(scales + r * blocks + b));
                const float f1 = b + 1 < blocks ? scale_value(__ldg(scales + r * blocks + b + 1)) : f0;
                const int split = static_cast<int>((b + 1) * BLOCK - first);  // elements of the first block
                float2 v[E / 2];
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    float2 q[2];
                    unpack_int8x4(q, u[i]);
                    v[2 * i] = make_float2(q[0].x * (4 * i < split ? f0 : f1), q[0].y * (4 * i + 1 < split ? f0 : f1));
                    v[2 * i + 1] = make_float2(q[1].x * (4 * i + 2 < split ? f0 : f1), q[1].y * (4 * i + 3 < split ? f0 : f1));
                }
                if (skip == 0 && c + E <= cols) {
                    store_vec<T, E>(row + c, v);
                } else {
                    const int n = static_cast<int>(cols - first < E - skip ? cols - first : E - skip);
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (i < n) from_float(row[first + i], i % 2 ? v[i / 2].y : v[i / 2].x);
                }
            }
        }
    }
}

// Threads side by side, and the grid: eight blocks to an SM at most, which stay and go down the rows.
template <typename F>
int by_rows(int64_t rows, int64_t spans, F&& start)
{
    int lanes_log2 = 2;
    while (lanes_log2 < 8 && (int64_t(1) << lanes_log2) < spans) ++lanes_log2;
    const int64_t across = cdiv<int64_t>(spans, int64_t(1) << lanes_log2), down = cdiv<int64_t>(rows, (I_THREADS >> lanes_log2) * I_DEPTH);
    const int64_t most = cdiv<int64_t>(SMS * 8, across) < 65535 ? cdiv<int64_t>(SMS * 8, across) : 65535;
    if (across > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    return start(dim3(static_cast<unsigned>(across), static_cast<unsigned>(down < most ? down : most)), lanes_log2) == cudaSuccess ? CONV2D_OK
                                                                                                                                  : CONV2D_ERR_CUDA;
}

template <typename T>
int quantize_int8(const void* x, uint8_t* data, uint8_t* scales, int64_t rows, int64_t cols, int64_t x_stride, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool vec = cols % V == 0 && (x_stride % V == 0 || rows == 1) && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    return by_rows(rows, cdiv<int64_t>(cols, BLOCK) * (BLOCK / SPAN<T>), [&](dim3 grid, int lanes_log2) {
        return launch(vec ? quantize_int8<T, true> : quantize_int8<T, false>, grid, I_THREADS, 0, stream, 1, static_cast<const T*>(x), data, scales,
                      rows, cols, x_stride, lanes_log2);
    });
}

template <typename T>
int dequantize_int8(const uint8_t* data, const uint8_t* scales, void* y, int64_t rows, int64_t cols, cudaStream_t stream)
{
    constexpr int V = 16 / sizeof(T);
    const bool vec = cols % V == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
    return by_rows(rows, cdiv<int64_t>(cols + (vec ? 0 : V - 1), SPAN<T>), [&](dim3 grid, int lanes_log2) {
        return launch(vec ? dequantize_int8<T, true> : dequantize_int8<T, false>, grid, I_THREADS, 0, stream, 1, data, scales, static_cast<T*>(y),
                      rows, cols, lanes_log2);
    });
}

}  // namespace mx
}  // namespace sgb

using namespace sgb;

extern "C" size_t mxint8_data_bytes(int64_t rows, int64_t cols)
{
    if (!mx::int8_extents_ok(rows, cols)) return 0;
    return static_cast<size_t>(rows) * static_cast<size_t>(mx::cdiv<int64_t>(cols, mx::BLOCK)) * mx::BLOCK;
}

extern "C" size_t mxint8_scale_bytes(int64_t rows, int64_t cols)
{
    if (!mx::int8_extents_ok(rows, cols)) return 0;
    return static_cast<size_t>(rows) * static_cast<size_t>(mx::cdiv<int64_t>(cols, mx::BLOCK));
}

extern "C" int mxint8_quantize(int64_t rows, int64_t cols, const void* x_dev, int32_t x_dtype, int64_t x_stride, void* data_dev,
                               void* scales_dev, conv2d_stream_t stream)
{
    if (rows < 0 || cols < 1 || x_stride < cols || (x_dtype != CONV2D_OUT_F32 && x_dtype != CONV2D_OUT_BF16)) return CONV2D_ERR_INVALID;
    if (rows > mx::INT8_MOST || cols > mx::INT8_MOST) return CONV2D_ERR_UNSUPPORTED;
    if (rows == 0) return CONV2D_OK;
    if (!x_dev || !data_dev || !scales_dev) return CONV2D_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(data_dev) % 16 || reinterpret_cast<uintptr_t>(x_dev) % (x_dtype == CONV2D_OUT_BF16 ? 2 : 4))
        return CONV2D_ERR_ALIGNMENT;
    uint8_t *d = static_cast<uint8_t*>(data_dev), *s = static_cast<uint8_t*>(scales_dev);
    return x_dtype == CONV2D_OUT_BF16 ? mx::quantize_int8<__nv_bfloat16>(x_dev, d, s, rows, cols, x_stride, stream)
                                      : mx::quantize_int8<float>(x_dev, d, s, rows, cols, x_stride, stream);
}

extern "C" int mxint8_dequantize(int64_t rows, int64_t cols, const void* data_dev, const void* scales_dev, void* y_dev,
                                 int32_t y_dtype, conv2d_stream_t stream)
{
    if (rows < 0 || cols < 1 || (y_dtype != CONV2D_OUT_F32 && y_dtype != CONV2D_OUT_BF16)) return CONV2D_ERR_INVALID;
    if (rows > mx::INT8_MOST || cols > mx::INT8_MOST) return CONV2D_ERR_UNSUPPORTED;
    if (rows == 0) return CONV2D_OK;
    if (!data_dev || !scales_dev || !y_dev) return CONV2D_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(data_dev) % 16 || reinterpret_cast<uintptr_t>(y_dev) % (y_dtype == CONV2D_OUT_BF16 ? 2 : 4))
        return CONV2D_ERR_ALIGNMENT;
    const uint8_t *d = static_cast<const uint8_t*>(data_dev), *s = static_cast<const uint8_t*>(scales_dev);
    return y_dtype == CONV2D_OUT_BF16 ? mx::dequantize_int8<__nv_bfloat16>(d, s, y_dev, rows, cols, stream)
                                      : mx::dequantize_int8<float>(d, s, y_dev, rows, cols, stream);
}
