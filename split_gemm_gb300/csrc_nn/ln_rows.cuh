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

template <int G>
constexpr int block_threads() { return G <= 32 ? 256 : G; }


// VEC elements as they lie in memory: one load or store of up to 16 bytes, two where fp32 elements make 32.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ void load(Pack<T, VEC>& d, const T* p)
{
    d = *reinterpret_cast<const Pack<T, VEC>*>(p);
}

template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const Pack<T, VEC>& d)
{
    *reinterpret_cast<Pack<T, VEC>*>(p) = d;
}

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
__global__ void __launch_bounds__(block_threads<G>()) fwd_rows(const TX* __restrict__ x, TY* y, const FwdParams p)
{
    constexpr bool MX = std::is_same_v<TY, void>;
    constexpr int NV = E / VEC, ROWS = block_threads<G>() / G;
    static_assert(!MX || (VEC == 1 ? G >= 32 : G * VEC >= 128), "four blocks' scales are joined within a row's lanes");
    constexpr bool HOLD = G * E <= 8192;  // weight and bias in registers; a wider row's block has no room for them
    __shared__ float sums[2][1][32];
    const int t = threadIdx.x % G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t end = MX ? p.padded_rows : p.rows;
    // rows of a warp run together, so that shuffles have all lanes
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int64_t lead = G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / G : first;
    const int blocks = MX ? mx::cdiv(p.cols, mx::BLOCK) : 0, btiles = MX ? mx::cdiv(blocks, mx::TILE_BLOCKS) : 0;

    float w[HOLD ? E : 1], b[HOLD ? E : 1];
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = (i / VEC * G + t) * VEC + i % VEC;
            w[i] = p.weight && c < p.cols ? p.weight[c] : 1.f;
            b[i] = p.bias && c < p.cols ? p.bias[c] : 0.f;
        }
    }
    Pack<TX, VEC> next[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * G + t) * VEC;
            if (r < p.rows && c < p.cols) load(next[k], x + r * p.x_stride + c);
        }
    };
    fetch(first);
    for (int64_t r = first, r_lead = lead; r_lead < end; r += step, r_lead += step) {
        Pack<TX, VEC> row[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) row[k] = next[k];
        fetch(r + step);
        const bool live = r < p.rows;
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i)
            if ((i / VEC * G + t) * VEC < p.cols) s[0] += mx::to_float(row[i / VEC].v[i % VEC]);
        row_sum<G>(s, sums[0]);
        const float mean = s[0] * p.inv_cols;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if ((i / VEC * G + t) * VEC < p.cols) {
                const float d = mx::to_float(row[i / VEC].v[i % VEC]) - mean;
                s[0] = fmaf(d, d, s[0]);
            }
        row_sum<G>(s, sums[1]);
        const float rstd = 1.f / sqrtf(s[0] * p.inv_cols + p.eps);
        if (live && t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * G + t) * VEC;
            const bool in = live && c < p.cols;
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float wi, bi;
                if constexpr (HOLD) {
                    wi = w[k * VEC + i];
                    bi = b[k * VEC + i];
                } else {
                    wi = p.weight && in ? __ldg(p.weight + c + i) : 1.f;
                    bi = p.bias && in ? __ldg(p.bias + c + i) : 0.f;
                }
                v[i] = in ? fmaf((mx::to_float(row[k].v[i]) - mean) * rstd, wi, bi) : 0.f;
            }
            if constexpr (MX) {
                store_mx<VEC>(v, r, c, p, live ? blocks : 0, blocks, r < end ? btiles : 0);
            } else if (in) {
                Pack<TY, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) mx::from_float(o.v[i], v[i]);
                store(y + r * p.y_stride + c, o);
            }
        }
    }
}

// Backward: dx, and this block's part of dweight and dbias.
template <typename TX, typename TY, int VEC, int E, int G>
__global__ void __launch_bounds__(block_threads<G>()) bwd_rows(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                               TX* __restrict__ dx, const BwdParams p)
{
    constexpr int NV = E / VEC, THREADS_ = block_threads<G>(), ROWS = THREADS_ / G;
    __shared__ float sums[2][2][32];
    __shared__ float join[G <= 32 ? 2 * G * E : 1];
    const int t = threadIdx.x % G;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / G;
    const int64_t lead = G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / G : first;

    float w[E], dw[E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = (i / VEC * G + t) * VEC + i % VEC;
        w[i] = p.weight && c < p.cols ? p.weight[c] : 1.f;
        dw[i] = db[i] = 0.f;
    }
    Pack<TX, VEC> next_x[NV];
    Pack<TY, VEC> next_g[NV];
    float next_mean = 0.f, next_rstd = 0.f;
    auto fetch = [&](int64_t r) {
        if (r < p.rows) {
            next_mean = __ldg(p.mean + r);
            next_rstd = __ldg(p.rstd + r);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * G + t) * VEC;
            if (r < p.rows && c < p.cols) {
                load(next_x[k], x + r * p.x_stride + c);
                load(next_g[k], dy + r * p.dy_stride + c);
            }
        }
    };
    fetch(first);
    int flip = 0;
    for (int64_t r = first, r_lead = lead; r_lead < p.rows; r += step, r_lead += step, flip ^= 1) {
        Pack<TX, VEC> row[NV];
        Pack<TY, VEC> grad[NV];
        const float mean = next_mean, rstd = next_rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            row[k] = next_x[k];
            grad[k] = next_g[k];
        }
        fetch(r + step);
        const bool live = r < p.rows;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (live && (i / VEC * G + t) * VEC < p.cols) {
                const float d = mx::to_float(grad[i / VEC].v[i % VEC]);
                const float xh = (mx::to_float(row[i / VEC].v[i % VEC]) - mean) * rstd;
                const float g = d * w[i];
                s[0] += g;
                s[1] = fmaf(g, xh, s[1]);
                dw[i] = fmaf(d, xh, dw[i]);
                db[i] += d;
            }
        row_sum<G>(s, sums[flip]);
        s[0] *= p.inv_cols;
        s[1] *= p.inv_cols;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * G + t) * VEC;
            if (!live || c >= p.cols) continue;
            Pack<TX, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float xh = (mx::to_float(row[k].v[i]) - mean) * rstd;
                mx::from_float(o.v[i], rstd * (fmaf(mx::to_float(grad[k].v[i]), w[k * VEC + i], -s[0]) - xh * s[1]));
            }
            store(dx + r * p.cols + c, o);
        }
    }
    if (!p.part) return;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
    if constexpr (G <= 32) {
        // the warp's rows by shuffles, then the warps one after another
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int o = G; o < 32; o <<= 1) {
                dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
                db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
            }
        for (int turn = 0; turn < THREADS_ / 32; ++turn) {
            if (static_cast<int>(threadIdx.x >> 5) == turn && (threadIdx.x & 31) < G) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int at = i * G + t;
                    join[at] = turn ? join[at] + dw[i] : dw[i];
                    join[G * E + at] = turn ? join[G * E + at] + db[i] : db[i];
                }
            }
            __syncthreads();
        }
        for (int at = threadIdx.x; at < G * E; at += THREADS_) {
            const int i = at / G, c = (i / VEC * G + at % G) * VEC + i % VEC;
            if (c < p.cols) {
                part[c] = join[at];
                part[p.cols + c] = join[G * E + at];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = (i / VEC * G + t) * VEC + i % VEC;
            if (c < p.cols) {
                part[c] = dw[i];
                part[p.cols + c] = db[i];
            }
        }
    }
}

}  // namespace ln
}  // namespace sgb
