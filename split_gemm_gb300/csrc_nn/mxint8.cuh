// The MXINT8 format on the device (OCP Microscaling Formats v1.0: 8-bit integers in blocks of 32 with an E8M0 scale), and
// reading of rows that begin anywhere.
#pragma once

#include "mx_common.cuh"
#include "ptx.cuh"

namespace sgb {
namespace mx {

// Scale byte of a block from the largest absolute value's fp32 bits: the biased exponent, floor(log2) + 127, 0 for zeros and values
// below 2^-126, 255 for a NaN or an infinity (the bits of absolute values order like integers).
__device__ __forceinline__ uint32_t int8_scale_byte(uint32_t amax_bits) { return amax_bits >> 23; }

// 2^-e for scale byte e + 127; byte 254 gives 2^-127, a subnormal number.  A NaN block's integers do not matter.
__device__ __forceinline__ float int8_inverse(uint32_t byte) { return __uint_as_float(byte >= 254u ? 0x00400000u : (254u - byte) << 23); }

// Four values, scaled to (-2, 2), to integers of 64ths: nearest even by adding 1.5 * 2^23 (the product by 64 is exact), in four bytes.
__device__ __forceinline__ uint32_t pack_int8x4(float a, float b, float c, float d)
{
    constexpr float MAGIC = 12582912.f;
    // saturation of what rounds to 128 in value: 127 and a half is where rounding leaves 127
    auto one = [&](float v) { return __float_as_uint(fminf(fmaxf(fmaf(v, 64.f, MAGIC), MAGIC - 127.f), MAGIC + 127.f)); };
    const uint32_t lo = __byte_perm(one(a), one(b), 0x0040), hi = __byte_perm(one(c), one(d), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// The integers of a word as floats over 64 (exact): xor 0x80 makes the byte q + 128 an unsigned one, which as the low mantissa byte of
// 2^17 + ... counts 64ths.
__device__ __forceinline__ void unpack_int8x4(float2 (&v)[2], uint32_t word)
{
    const uint32_t u = word ^ 0x80808080u;
    constexpr uint32_t BASE = 0x48000000u;         // 2^17: its last bit counts 2^-6
    constexpr float MINUS = -131074.f;             // -(2^17 + 128/64)
    v[0] = add2(make_float2(__uint_as_float(__byte_perm(u, BASE, 0x7650)), __uint_as_float(__byte_perm(u, BASE, 0x7651))), make_float2(MINUS, MINUS));
    v[1] = add2(make_float2(__uint_as_float(__byte_perm(u, BASE, 0x7652)), __uint_as_float(__byte_perm(u, BASE, 0x7653))), make_float2(MINUS, MINUS));
}

// N words from byte address p, which need not be aligned beyond `GRAIN` bytes, zero from byte `valid` on (a multiple of GRAIN).  Memory is read in
// aligned 16-byte vectors that hold at least one valid byte each, so nothing is touched outside the vectors of the row.
template <int N, int GRAIN>
__device__ __forceinline__ void load_any(uint32_t (&w)[N], const void* p, int valid)
{
    static_assert(N % 4 == 0);
    const int s = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* base = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) - s);
    uint32_t u[N + 4];
#pragma unroll
    for (int i = 0; i < N / 4 + 1; ++i) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (16 * i - s < valid && (i < N / 4 || s > 0)) q = __ldg(base + i);
        u[4 * i] = q.x;
        u[4 * i + 1] = q.y;
        u[4 * i + 2] = q.z;
        u[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < N + 2; ++i) u[i] = s & 8 ? u[i + 2] : u[i];
#pragma unroll
    for (int i = 0; i < N + 1; ++i) u[i] = s & 4 ? u[i + 1] : u[i];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t v = GRAIN >= 4 ? u[i] : __funnelshift_r(u[i], u[i + 1], 8 * (s & 3));
        const int left = valid - 4 * i;  // bytes of the word that count
        if (GRAIN >= 4)
            v = left > 0 ? v : 0u;
        else
            v = left >= 4 ? v : left <= 0 ? 0u : v & (0xffffffffu >> (32 - 8 * left));
        w[i] = v;
    }
}

}  // namespace mx
}  // namespace sgb
