// The MXFP4 format on the device (OCP Microscaling Formats v1.0: E2M1 elements,
// blocks of 32, E8M0 scales) and small helpers shared by the kernels of this folder.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace sgb {
namespace mx {

constexpr int SMS = 152;           // of a GB300
constexpr int BLOCK = 32;          // elements that share a scale
constexpr int TILE_ROWS = 128;     // scale tile: 128 rows x 4 blocks = 512 bytes
constexpr int TILE_BLOCKS = 4;
constexpr int TILE_BYTES = 512;

template <typename T>
__host__ __device__ constexpr T cdiv(T a, T b) { return a / b + (a % b != 0); }  // a up to the type's largest

// Byte of row r, block b within the scales of a matrix with `btiles` tiles to a row of tiles.
__host__ __device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t btiles)
{
    return ((r >> 7) * btiles + (b >> 2)) * TILE_BYTES + ((r & 31) << 4) + ((r & 127) >> 5 << 2) + (b & 3);
}

// Scale byte of a block from the largest absolute value's fp32 bits.  The biased
// exponent E is floor(log2) + 127, so the byte is E - 2, clamped at 0 (zeros and
// values below 2^-125); E = 255, which any NaN or infinity of the block gives
// because the bits of absolute values order like integers, marks the block as NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^-e for scale byte e + 127: always a normal number (the byte is at most 252).
// A NaN block's elements are stored as they come (their scale makes them NaN).
__device__ __forceinline__ float inverse_scale(uint32_t byte)
{
    return __uint_as_float((byte == 255u ? 127u : 254u - byte) << 23);
}

// 2^e; byte 0 is 2^-127, a subnormal number, and byte 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}

// The largest of three absolute values; NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Eight fp32 values to E2M1 (nearest even, saturating), the first in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The values of four bytes' eight E2M1 codes, the lowest first (exact: E2M1 values are fp16 numbers).
__device__ __forceinline__ void unpack_e2m1x8(float2 (&v)[4], uint32_t word)
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(word));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float& d, float v) { d = v; }
__device__ __forceinline__ void from_float(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Launches a kernel that may get ready while the one before it on the stream ends; it waits for that one itself
// (griddepcontrol.wait) before it touches global memory.  cluster > 1: in clusters of so many blocks.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, int cluster, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, int smem, cudaStream_t stream, int cluster, A... args)
{
    return launch(kernel, dim3(static_cast<unsigned>(grid)), threads, smem, stream, cluster, args...);
}

// Lets a kernel have `bytes` of dynamic shared memory; asked of the driver once per device.
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done)
{
    if (bytes <= 40 * 1024) return true;  // 48 KB with the static arrays needs no asking
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev < 64) done.fetch_or(bit, std::memory_order_release);
    return true;
}

}  // namespace mx
}  // namespace sgb
