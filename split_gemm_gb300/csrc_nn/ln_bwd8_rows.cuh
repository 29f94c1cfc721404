// The norm's gradient with x as an 8-bit checkpoint, rows held in registers: the kernels of ln_rows.cuh (bwd_rows) with another x.
//
// A thread's vectors are 8 elements: 8 bytes of the checkpoint, 16 or 32 of dy and dx.  Both come through rings that a thread alone reads; the scale byte
// of each vector's block comes a row ahead in a register.  Where dy's rows do not start at 16 bytes (WHOLE = false), `off` elements of the row before
// stand in front of dy's first vector; the checkpoint's rows always start at 32 bytes, so that the thread's 8 integers then lie `off` to the left, in two
// neighbouring 8-byte pieces and in one or two blocks.
//
// HBM binds, at 33/32 + 2 or 4 bytes read and 2 or 4 written for each element: 32768 x 4096, dy bf16, 140 us, 4.8 TB/s (the bf16 kernel of ln_rows.cuh
// takes 141 us for 19% more bytes).  What stands between are the conversions and the reductions of 16 warps an SM, as there; which of them was not told apart.
#pragma once

#include "ln_rows.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ln {

// A checkpoint's rows, of blocks * 32 bytes.
struct Checkpoint {
    const uint8_t *data, *scales;
    int64_t blocks;
    __device__ __forceinline__ float at(int64_t r, int64_t c) const
    {
        const int q = static_cast<int8_t>(__ldg(data + r * (blocks * mx::BLOCK) + c));
        return static_cast<float>(q) * 0.015625f * mx::scale_value(__ldg(scales + r * blocks + c / mx::BLOCK));
    }
};

// Bytes of both rings for a thread and a row: pieces of 8 bytes, two for each unaligned vector.
template <typename TY, int E, bool WHOLE>
constexpr int RING8 = E / 8 * (WHOLE ? 8 : 16) + E * static_cast<int>(sizeof(TY));

template <typename TY, int E, int G, int MOST, bool WHOLE>
constexpr int depth8()
{
    const int row = bwd_threads(RowShape{G ? G : MOST, E, MOST}) * RING8<TY, E, WHOLE>;
    const int n = 72 * 1024 / row;
    return n > 4 ? 4 : n >= 2 ? n : 2;
}

template <typename TY, int E, int G, int MOST, bool SUMS, bool WHOLE>
__global__ void __launch_bounds__(MOST, BWD_RESIDENT<G, E, MOST>) bwd8_rows(const TY* dy, const Checkpoint x, TY* dx, const BwdParams p)
{
    constexpr int VEC = 8, ROWS = G ? MOST / G : 1, DEPTH = depth8<TY, E, G, MOST, WHOLE>();
    using Un = Units<VEC, E, WHOLE>;
    constexpr int U = Un::U, H = Un::H;
    constexpr int PIECES = WHOLE ? 1 : 2;
    extern __shared__ __align__(16) uint8_t ring_mem[];
    __shared__ float sums[2][2][32];
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int group = G ? G : blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + (G ? threadIdx.x / (G ? G : 1) : 0);
    const int64_t lead = G && G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / (G ? G : 1) : first;
    const Un un(G ? threadIdx.x % (G ? G : 1) : threadIdx.x, group, WHOLE ? 0 : static_cast<int>(first * p.dy_stride % VEC), p.cols);
    const int pitch = static_cast<int>(x.blocks) * mx::BLOCK, off = un.off;

    using RingG = Ring<TY, VEC, Un::NV, DEPTH, false>;
    const RingG ring_g(ring_mem, blockDim.x);
    // the checkpoint's ring: [slot][vector][piece][thread] of 8 bytes
    uint8_t* const mine = ring_mem + RingG::THREAD_BYTES * blockDim.x + 8 * threadIdx.x;
    const int piece_pitch = 8 * blockDim.x;
    const auto piece_at = [&](int slot, int u, int j) { return mine + ((slot * U + u) * PIECES + j) * piece_pitch; };
    const auto ask = [&](int slot, int64_t r) {
        const bool live = r < p.rows;
        const int front = live ? off : 0;
        ring_g.ask(slot, dy + (live ? r * p.dy_stride : 0), un.t * VEC - front, group * VEC, live ? p.cols : 0, front);
        const uint8_t* row = x.data + (live ? r * pitch : 0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {  // of unaligned vectors the piece before, and the one at the vector's own number
                const int c = (u * group + un.t + (WHOLE ? 0 : j - 1)) * VEC;
                const bool in = live && c >= 0 && c < pitch;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(ptx::smem_addr(piece_at(slot, u, j))), "l"(in ? row + c : x.data), "r"(in ? 8 : 0)
                             : "memory");
            }
        ptx::cp_async_commit();
    };
    // Scale bytes of a row's vectors: of an unaligned one the blocks of its first and last element, which may differ.
    uint32_t scale[U];
    const auto scales_of = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = un.col(u, 0);
            const bool live = r < p.rows;
            const uint8_t* s = x.scales + (live ? r * x.blocks : 0);
            if constexpr (WHOLE) {
                scale[u] = live && c < pitch ? __ldg(s + c / mx::BLOCK) : 0u;
            } else {
                const int lo = c < 0 ? 0 : c, hi = c + 7;
                const uint32_t a = live && lo < pitch ? __ldg(s + lo / mx::BLOCK) : 0u;
                scale[u] = a | (live && hi < pitch && hi >= 0 && hi / mx::BLOCK != lo / mx::BLOCK ? __ldg(s + hi / mx::BLOCK) << 8 : a << 8);
            }
        }
    };
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) ask(k, first + k * step);
    float mean = first < p.rows ? __ldg(p.mean + first) : 0.f, rstd = first < p.rows ? __ldg(p.rstd + first) : 0.f;
    scales_of(first);

    float2 w[U][H], dw[SUMS ? U : 1][H], db[SUMS ? U : 1][H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        un.params(w[u], p.weight, u, 1.f);
        if constexpr (SUMS)
#pragma unroll
            for (int i = 0; i < H; ++i) dw[u][i] = db[u][i] = make_float2(0.f, 0.f);
    }
    const bool ragged = un.ragged();
    int slot = 0, flip = 0;
    for (int64_t r = first, r_lead = lead; r_lead < p.rows; r += step, r_lead += step, flip ^= 1) {
        // Lanes past the last row take a row of zeros, so that they add nothing.
        const bool live = r < p.rows;
        const float2 minus = make_float2(-mean, -mean), rs = make_float2(rstd, rstd);
        mean = r + step < p.rows ? __ldg(p.mean + r + step) : 0.f;
        rstd = r + step < p.rows ? __ldg(p.rstd + r + step) : 0.f;
        ptx::cp_async_wait<DEPTH - 1>();
        float2 xh[U][H], g[U][H];
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            un.template take<TY>(g[u], ring_g, slot, dy + r * p.dy_stride, u, live);
            uint2 q = *reinterpret_cast<const uint2*>(piece_at(slot, u, PIECES - 1));
            if constexpr (!WHOLE) {  // the vector's bytes begin `off` before its own piece
                const uint2 before = *reinterpret_cast<const uint2*>(piece_at(slot, u, 0));
                uint32_t v[4] = {before.x, before.y, q.x, q.y};
                const int skip = (8 - off) & 7;  // of the piece before; with off = 0 nothing of it counts
                if (off != 0) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) v[i] = skip & 4 ? v[i + 1] : v[i];
                    q.x = __funnelshift_r(v[0], v[1], 8 * (skip & 3));
                    q.y = __funnelshift_r(v[1], v[2], 8 * (skip & 3));
                }
            }
            float2 a[2], b[2];
            mx::unpack_int8x4(a, q.x);
            mx::unpack_int8x4(b, q.y);
            if constexpr (WHOLE) {
                const float f = mx::scale_value(scale[u]);
                xh[u][0] = mx::mul2(a[0], make_float2(f, f));
                xh[u][1] = mx::mul2(a[1], make_float2(f, f));
                xh[u][2] = mx::mul2(b[0], make_float2(f, f));
                xh[u][3] = mx::mul2(b[1], make_float2(f, f));
            } else {
                const float f0 = mx::scale_value(scale[u] & 255u), f1 = mx::scale_value(scale[u] >> 8);
                const int c = un.col(u, 0), split = mx::BLOCK - (c & (mx::BLOCK - 1));  // elements of the first block
                const auto f = [&](int i) { return c >= 0 && i >= split ? f1 : f0; };
                xh[u][0] = mx::mul2(a[0], make_float2(f(0), f(1)));
                xh[u][1] = mx::mul2(a[1], make_float2(f(2), f(3)));
                xh[u][2] = mx::mul2(b[0], make_float2(f(4), f(5)));
                xh[u][3] = mx::mul2(b[1], make_float2(f(6), f(7)));
            }
        }
        scales_of(r + step);
        // As in bwd_rows: outside the row dy is zero, and so is the checkpoint, or another row's integers in front of it; where a normalised zero may be past
        // fp32, the mean stands in x's place.
        un.cut(xh);
        un.cut(g);
        if (ragged && __any_sync(0xffffffffu, !(fabsf(minus.x * rs.x) <= FLT_MAX))) un.fill(xh, -minus.x);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                xh[u][i] = mul2(add2(xh[u][i], minus), rs);
                if constexpr (SUMS) {
                    dw[u][i] = fma2(g[u][i], xh[u][i], dw[u][i]);
                    db[u][i] = add2(db[u][i], g[u][i]);
                }
                g[u][i] = mul2(g[u][i], w[u][i]);
                s0 = add2(s0, g[u][i]);
                s1 = fma2(g[u][i], xh[u][i], s1);
            }
        }
        float s[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<G>(s, sums[flip]);
        ask(slot, r + DEPTH * step);  // what the slot held is in registers
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
        const float m0 = -s[0] * p.inv_cols, m1 = -s[1] * p.inv_cols;
        s0 = make_float2(m0, m0);
        s1 = make_float2(m1, m1);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) xh[u][i] = mul2(rs, fma2(xh[u][i], s1, add2(g[u][i], s0)));
        un.put(dx + r * p.cols, xh, live);
    }
    ptx::cp_async_wait_all();
    if constexpr (SUMS) {
        if (!p.part) return;
        float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
        auto at_w = [&](int i) -> float& { return i % 2 ? dw[i / 2 / H][i / 2 % H].y : dw[i / 2 / H][i / 2 % H].x; };
        auto at_b = [&](int i) -> float& { return i % 2 ? db[i / 2 / H][i / 2 % H].y : db[i / 2 / H][i / 2 % H].x; };
        auto col = [&](int i) { return un.col(i / (2 * H), i % (2 * H)); };
        if constexpr (G > 0) {
            // Each row's sums by column in shared memory (rows may have different `off`), then the rows in order.
            float* join = reinterpret_cast<float*>(ring_mem);
            constexpr int W = G * E;
            __syncthreads();  // the ring is done with
            float* row = join + threadIdx.x / (G ? G : 1) * W;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(i);
                if (static_cast<unsigned>(c) < static_cast<unsigned>(p.cols)) {
                    row[c] = at_w(i);
                    row[ROWS * W + c] = at_b(i);
                }
            }
            __syncthreads();
            for (int e = threadIdx.x; e < 2 * p.cols; e += MOST) {
                const bool second = e >= p.cols;
                const float* from = join + (second ? ROWS * W + e - p.cols : e);
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < ROWS; ++k) v += from[k * W];
                part[e] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(i);
                if (static_cast<unsigned>(c) < static_cast<unsigned>(p.cols)) {
                    part[c] = at_w(i);
                    part[p.cols + c] = at_b(i);
                }
            }
        }
    }
}

}  // namespace ln
}  // namespace sgb
