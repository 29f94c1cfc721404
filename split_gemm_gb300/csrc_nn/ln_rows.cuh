// Layer normalisation kernels that hold their row in registers: one reading of x.
//
// G threads share a row, each with E elements in E/VEC vectors; vector k of thread t is number k*G + t of the
// row, so neighbouring threads read neighbouring vectors.  G <= 32: a warp holds 32/G rows and sums by
// shuffles.  G >= 128: a block holds one row and sums through shared memory, one barrier to a sum.  Blocks
// stay for many rows: a thread's columns are the same in each, so weight and bias (forward, backward) and the
// sums of dweight and dbias (backward) stay in registers, and the next row is loaded before the current one is worked on.
//
// All of them are bound by HBM: per element the forward pass moves sizeof(x) + sizeof(y) bytes for about 8 operations.
#pragma once

#include <type_traits>

#include "ln_params.cuh"

namespace sgb {
namespace ln {


// VEC elements as they lie in memory: one load or store of up to 16 bytes, two where fp32 elements make 32.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

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

// How a thread's E elements are paired for two-wide arithmetic: a unit is a vector, or two single elements G apart.
template <int VEC, int E, int G>
struct Units {
    static constexpr int U = VEC > 1 ? E / VEC : E / 2;  // units of a thread
    static constexpr int H = VEC > 1 ? VEC / 2 : 1;      // pairs of a unit
    static constexpr int NV = E / VEC;
    int t;
    // column of element i of unit u
    __device__ __forceinline__ int col(int u, int i) const { return VEC > 1 ? (u * G + t) * VEC + i : (2 * u + i) * G + t; }
    template <typename T>
    __device__ __forceinline__ void widen(float2 (&d)[H], const Pack<T, VEC> (&v)[NV], int u) const
    {
        if constexpr (VEC == 1) {
            d[0] = make_float2(mx::to_float(v[2 * u].v[0]), mx::to_float(v[2 * u + 1].v[0]));
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[u]);
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = make_float2(v[u].v[2 * i], v[u].v[2 * i + 1]);
        }
    }
    // Stores a unit's values at columns below `cols` of `row`.
    template <typename T>
    __device__ __forceinline__ void store_unit(T* row, const float2 (&d)[H], int u, int cols) const
    {
        if constexpr (VEC == 1) {
            if (col(u, 0) < cols) mx::from_float(row[col(u, 0)], d[0].x);
            if (col(u, 1) < cols) mx::from_float(row[col(u, 1)], d[0].y);
        } else if (col(u, 0) < cols) {
            Pack<T, VEC> o;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(d[i].x, d[i].y);
                    o.v[2 * i] = b.x;
                    o.v[2 * i + 1] = b.y;
                } else {
                    o.v[2 * i] = d[i].x;
                    o.v[2 * i + 1] = d[i].y;
                }
            }
            *reinterpret_cast<Pack<T, VEC>*>(row + col(u, 0)) = o;
        }
    }
    // A unit's values of a per-column fp32 vector (`other` where there is none).
    __device__ __forceinline__ void params(float2 (&d)[H], const float* v, int u, int cols, float other) const
    {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int c0 = col(u, 2 * i), c1 = col(u, 2 * i + 1);
            d[i] = make_float2(v && c0 < cols ? __ldg(v + c0) : other, v && c1 < cols ? __ldg(v + c1) : other);
        }
    }
    template <typename T>
    __device__ __forceinline__ void fetch(Pack<T, VEC> (&d)[NV], const T* row, bool live, int cols) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * G + t) * VEC;
            if (live && c < cols)
                d[k] = *reinterpret_cast<const Pack<T, VEC>*>(row + c);
            else
                d[k] = Pack<T, VEC>{};
        }
    }
};

// Sums over the G threads of a row; `buf` is a buffer that no thread reads any more.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[32])
{
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (G > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = buf[i][lane & (G / 32 - 1)];
#pragma unroll
        for (int o = G / 64; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// Stores one vector's values as part of a quantised row (all lanes of a warp take part): the 32/VEC lanes that
// hold a block of 32 share its scale.  Elements are stored for blocks below `live`, scale bytes for the row's first `btiles` scale tiles.
template <int VEC>
__device__ __forceinline__ void store_mx(const float (&v)[VEC], int64_t r, int col, const FwdParams& p, int live, int blocks,
                                         int btiles)
{
    constexpr int LANES = mx::BLOCK / VEC;
    const int lane = threadIdx.x & 31;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = max(m, mx::abs_bits(v[i]));
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t byte = mx::scale_byte(m);
    const float inv = mx::inverse_scale(byte);
    const int b = col / mx::BLOCK;
    const bool in_data = b < live, in_tile = b < btiles * mx::TILE_BLOCKS;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = i < VEC ? v[i < VEC ? i : 0] * inv : 0.f;
    uint32_t word = mx::pack_e2m1x8(q);
    uint8_t* data = p.data + r * (static_cast<int64_t>(blocks) * 16) + col / 2;
    if constexpr (VEC == 8) {
        if (in_data) *reinterpret_cast<uint32_t*>(data) = word;
    } else if constexpr (VEC == 4) {
        if (in_data) *reinterpret_cast<uint16_t*>(data) = static_cast<uint16_t>(word);
    } else {  // one element to a lane: eight lanes' codes make a word
        word |= __shfl_xor_sync(0xffffffffu, word, 1) << 4;  // right in even lanes
        word |= __shfl_xor_sync(0xffffffffu, word, 2) << 8;
        word |= __shfl_xor_sync(0xffffffffu, word, 4) << 16;
        if (in_data && lane % 8 == 0) *reinterpret_cast<uint32_t*>(data) = word;
    }
    if constexpr (VEC == 1) {
        if (in_tile && lane == 0) p.scales[mx::scale_at(r, b, btiles)] = static_cast<uint8_t>(byte);
    } else {  // four blocks' bytes side by side
        uint32_t w = byte << (8 * (b & 3));
        w |= __shfl_xor_sync(0xffffffffu, w, LANES);
        w |= __shfl_xor_sync(0xffffffffu, w, 2 * LANES);
        if (in_tile && lane % (4 * LANES) == 0) *reinterpret_cast<uint32_t*>(p.scales + mx::scale_at(r, b, btiles)) = w;
    }
}

// Forward.  TY = void: the result quantised; rows from p.rows to p.padded_rows are the scale tiles' padding.
template <typename TX, typename TY, int VEC, int E, int G>
__global__ void __launch_bounds__(block_threads(G), fwd_resident({G, E})) fwd_rows(const TX* __restrict__ x, TY* y, const FwdParams p)
{
    constexpr bool MX = std::is_same_v<TY, void>;
    constexpr int ROWS = block_threads(G) / G;
    static_assert(!MX || (VEC == 1 ? G >= 32 : G * VEC >= 128), "four blocks' scales are joined within a row's lanes");
    constexpr bool HOLD = G * E <= 8192;  // weight and bias in registers; a wider row's block has no room for them
    using Un = Units<VEC, E, G>;
    constexpr int U = Un::U, H = Un::H;
    __shared__ float sums[2][1][32];
    const Un un{static_cast<int>(threadIdx.x) % G};
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t end = MX ? p.padded_rows : p.rows;
    // rows of a warp run together, so that shuffles have all lanes
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int64_t lead = G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / G : first;
    const int blocks = MX ? mx::cdiv(p.cols, mx::BLOCK) : 0, btiles = MX ? mx::cdiv(blocks, mx::TILE_BLOCKS) : 0;

    float2 w[HOLD ? U : 1][H], b[HOLD ? U : 1][H];
    if constexpr (HOLD) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            un.params(w[u], p.weight, u, p.cols, 1.f);
            un.params(b[u], p.bias, u, p.cols, 0.f);
        }
    }
    Pack<TX, VEC> next[Un::NV];
    un.fetch(next, x + first * p.x_stride, first < p.rows, p.cols);
    for (int64_t r = first, r_lead = lead; r_lead < end; r += step, r_lead += step) {
        const bool live = r < p.rows;
        float2 d[U][H];
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            un.widen(d[u], next, u);  // zeros beyond the row
#pragma unroll
            for (int i = 0; i < H; ++i) s2 = add2(s2, d[u][i]);
        }
        un.fetch(next, x + (r + step) * p.x_stride, r + step < p.rows, p.cols);
        float s[1] = {s2.x + s2.y};
        row_sum<G>(s, sums[0]);
        const float mean = s[0] * p.inv_cols;
        const float2 minus = make_float2(-mean, -mean);
        s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (un.col(u, 0) < p.cols) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    d[u][i] = add2(d[u][i], minus);
                    if (VEC == 1 && un.col(u, 1) >= p.cols) d[u][i].y = 0.f;
                    s2 = fma2(d[u][i], d[u][i], s2);
                }
            }
        s[0] = s2.x + s2.y;
        row_sum<G>(s, sums[1]);
        const float rstd = rsqrtf(s[0] * p.inv_cols + p.eps);
        if (live && un.t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
        const float2 scale = make_float2(rstd, rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (!HOLD) {
                un.params(w[0], p.weight, u, p.cols, 1.f);
                un.params(b[0], p.bias, u, p.cols, 0.f);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) d[u][i] = fma2(mul2(d[u][i], scale), w[HOLD ? u : 0][i], b[HOLD ? u : 0][i]);
            if constexpr (!MX) {
                un.store_unit(y + r * p.y_stride, d[u], u, live ? p.cols : 0);
            } else if constexpr (VEC == 1) {
                const float v0[1] = {live && un.col(u, 0) < p.cols ? d[u][0].x : 0.f};
                const float v1[1] = {live && un.col(u, 1) < p.cols ? d[u][0].y : 0.f};
                store_mx<1>(v0, r, un.col(u, 0), p, live ? blocks : 0, blocks, r < end ? btiles : 0);
                store_mx<1>(v1, r, un.col(u, 1), p, live ? blocks : 0, blocks, r < end ? btiles : 0);
            } else {
                const bool in = live && un.col(u, 0) < p.cols;
                float v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = in ? (i % 2 ? d[u][i / 2].y : d[u][i / 2].x) : 0.f;
                store_mx<VEC>(v, r, un.col(u, 0), p, live ? blocks : 0, blocks, r < end ? btiles : 0);
            }
        }
    }
}

// Backward: dx, and this block's part of dweight and dbias.
template <typename TX, typename TY, int VEC, int E, int G>
__global__ void __launch_bounds__(block_threads(G), bwd_resident({G, E})) bwd_rows(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                                                  TX* __restrict__ dx, const BwdParams p)
{
    constexpr int THREADS_ = block_threads(G), ROWS = THREADS_ / G;
    using Un = Units<VEC, E, G>;
    constexpr int U = Un::U, H = Un::H;
    __shared__ float sums[2][2][32];
    __shared__ float join[G <= 32 ? 2 * G * E : 1];
    const Un un{static_cast<int>(threadIdx.x) % G};
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int64_t lead = G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / G : first;

    float2 w[U][H], dw[U][H], db[U][H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        un.params(w[u], p.weight, u, p.cols, 1.f);
#pragma unroll
        for (int i = 0; i < H; ++i) dw[u][i] = db[u][i] = make_float2(0.f, 0.f);
    }
    Pack<TX, VEC> next_x[Un::NV];
    Pack<TY, VEC> next_g[Un::NV];
    float next_mean = 0.f, next_rstd = 0.f;
    auto fetch = [&](int64_t r) {
        const bool live = r < p.rows;
        if (live) {
            next_mean = __ldg(p.mean + r);
            next_rstd = __ldg(p.rstd + r);
        }
        un.fetch(next_x, x + r * p.x_stride, live, p.cols);
        un.fetch(next_g, dy + r * p.dy_stride, live, p.cols);
    };
    fetch(first);
    int flip = 0;
    for (int64_t r = first, r_lead = lead; r_lead < p.rows; r += step, r_lead += step, flip ^= 1) {
        // Lanes past the last row take a row of zeros, so that they add nothing.
        const bool live = r < p.rows;
        const float mean = live ? next_mean : 0.f, rstd = live ? next_rstd : 0.f;
        const float2 minus = make_float2(-mean, -mean), scale = make_float2(rstd, rstd);
        float2 xh[U][H], g[U][H];
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            un.widen(xh[u], next_x, u);
            un.widen(g[u], next_g, u);
            if (un.col(u, 0) < p.cols) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    xh[u][i] = mul2(add2(xh[u][i], minus), scale);
                    if (VEC == 1 && un.col(u, 1) >= p.cols) xh[u][i].y = 0.f;
                    dw[u][i] = fma2(g[u][i], xh[u][i], dw[u][i]);
                    db[u][i] = add2(db[u][i], g[u][i]);
                    g[u][i] = mul2(g[u][i], w[u][i]);
                    s0 = add2(s0, g[u][i]);
                    s1 = fma2(g[u][i], xh[u][i], s1);
                }
            }
        }
        fetch(r + step);
        float s[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<G>(s, sums[flip]);
        const float m0 = -s[0] * p.inv_cols, m1 = -s[1] * p.inv_cols;
        s0 = make_float2(m0, m0);
        s1 = make_float2(m1, m1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < H; ++i) xh[u][i] = mul2(scale, fma2(xh[u][i], s1, add2(g[u][i], s0)));
            un.store_unit(dx + r * p.cols, xh[u], u, live ? p.cols : 0);
        }
    }
    if (!p.part) return;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
    auto at_w = [&](int i) -> float& { return i % 2 ? dw[i / 2 / H][i / 2 % H].y : dw[i / 2 / H][i / 2 % H].x; };
    auto at_b = [&](int i) -> float& { return i % 2 ? db[i / 2 / H][i / 2 % H].y : db[i / 2 / H][i / 2 % H].x; };
    auto col = [&](int i, int t) { return Un{t}.col(i / (2 * H), i % (2 * H)); };  // of a thread's element i
    if constexpr (G <= 32) {
        // the warp's rows by shuffles, then the warps one after another
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int o = G; o < 32; o <<= 1) {
                at_w(i) += __shfl_xor_sync(0xffffffffu, at_w(i), o);
                at_b(i) += __shfl_xor_sync(0xffffffffu, at_b(i), o);
            }
        for (int turn = 0; turn < THREADS_ / 32; ++turn) {
            if (static_cast<int>(threadIdx.x >> 5) == turn && (threadIdx.x & 31) < G) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int at = i * G + un.t;
                    join[at] = turn ? join[at] + at_w(i) : at_w(i);
                    join[G * E + at] = turn ? join[G * E + at] + at_b(i) : at_b(i);
                }
            }
            __syncthreads();
        }
        for (int at = threadIdx.x; at < G * E; at += THREADS_) {
            const int c = col(at / G, at % G);
            if (c < p.cols) {
                part[c] = join[at];
                part[p.cols + c] = join[G * E + at];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = col(i, un.t);
            if (c < p.cols) {
                part[c] = at_w(i);
                part[p.cols + c] = at_b(i);
            }
        }
    }
}

}  // namespace ln
}  // namespace sgb
