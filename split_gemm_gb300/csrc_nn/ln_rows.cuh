// Layer normalisation kernels that hold their row in registers: one reading of x.
//
// A group of threads shares a row, each with E elements in E/VEC vectors of 16 bytes of x; vector k of thread t is
// number k*(group) + t of the row, so neighbouring threads read neighbouring vectors.  G = 4 .. 32: groups of G, a warp holds
// 32/G rows and sums by shuffles.  G = 0: a block of as many warps as the row needs holds one row and sums through shared
// memory, one barrier to a sum.  Blocks stay for many rows: a thread's columns are the same in each, so weight and bias (forward, backward) and the sums of
// dweight and dbias (backward) stay in registers.
//
// Rows come by cp.async into a ring of DEPTH rows in shared memory, in which a thread reads only what it asked for
// itself: no barrier belongs to the ring, and no register waits for memory.
//
// Rows that do not start at 16 bytes are read in whole vectors all the same: `off` elements of the row before
// stand in front of the first one, and are left out.  A group's rows lie a multiple of VEC rows apart, so `off`, and with it a thread's
// columns, is the same in all of them.  A row's end is cut off by the copy itself.
//
// Rows of whole vectors are bound by HBM, forward and (up to 8192 columns) backward: per element the forward pass moves
// sizeof(x) + sizeof(y) bytes for about 8 operations.  32768 x 4096 bf16: forward 90 us, 6.0 TB/s; backward 141 us, 5.7 TB/s.  Others are not:
// unaligned rows wait for their barriers and edges (16384 x 8191 bf16 142 us forward, 3.8 TB/s), and the quantised norm, which
// writes a quarter of the bytes, takes longer than the norm (16384 x 4096 bf16 53 us, 3.2 TB/s, against 44): for the instructions
// after the norm or for its scale bytes, each stored alone into sectors that rows of other blocks share; which was not told apart.
#pragma once

#include <cfloat>
#include <type_traits>

#include "ln_params.cuh"
#include "ptx.cuh"
#include "row_copy.h"

namespace sgb {
namespace ln {

template <int G, int E, int MOST>
constexpr int FWD_RESIDENT = fwd_resident(RowShape{G ? G : MOST, E, MOST});
template <int G, int E, int MOST>
constexpr int BWD_RESIDENT = bwd_resident(RowShape{G ? G : MOST, E, MOST});

// VEC elements as they lie in memory.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

using mx::add2;
using mx::fma2;
using mx::mul2;

// The rows on their way to a thread: DEPTH slots of NV vectors, 8 or 16 bytes to a copy.  WHOLE: rows are whole vectors.
template <typename T, int VEC, int NV, int DEPTH, bool WHOLE>
struct Ring {
    static constexpr int CHUNK = VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16, CHUNKS = VEC * sizeof(T) / CHUNK;
    static constexpr int PER = CHUNK / sizeof(T);  // elements of a copy
    static constexpr int THREAD_BYTES = DEPTH * NV * CHUNKS * CHUNK;
    uint8_t* mine;
    int pitch;  // bytes between a thread's chunks: a chunk of every thread
    __device__ __forceinline__ Ring(uint8_t* base, int threads) : mine(base + threadIdx.x * CHUNK), pitch(threads * CHUNK) {}
    __device__ __forceinline__ uint8_t* at(int slot, int k, int j) const { return mine + ((slot * NV + k) * CHUNKS + j) * pitch; }
    // Asks for the vectors at columns c0 + k*step of `row`, which begins `front` elements behind a whole vector's start; for no
    // row, `cols` and `front` are 0 and `row` is any aligned address.
    __device__ __forceinline__ void ask(int slot, const T* row, int c0, int step, int cols, int front) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
                const RowCopy copy = row_copy(c0 + k * step + j * PER, PER, cols, front, WHOLE);
                const int bytes = copy.count * static_cast<int>(sizeof(T));
                const T* src = row + copy.at;
                if constexpr (CHUNK == 16)
                    ptx::cp_async_16(at(slot, k, j), src, bytes);
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(ptx::smem_addr(at(slot, k, j))), "l"(src), "r"(bytes)
                                 : "memory");
            }
    }
    __device__ __forceinline__ void get(Pack<T, VEC>& d, int slot, int k) const
    {
        static_assert(CHUNK == 8 || CHUNK == 16);
        if constexpr (CHUNK == 8) {
            *reinterpret_cast<uint2*>(&d) = *reinterpret_cast<const uint2*>(at(slot, k, 0));
        } else {
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) reinterpret_cast<uint4*>(&d)[j] = *reinterpret_cast<const uint4*>(at(slot, k, j));
        }
    }
};

// A thread's E elements of a row as units of H pairs for two-wide arithmetic: a unit is a vector, or (VEC = 1) two
// single elements a group apart.  WHOLE: rows are whole vectors, so that a unit lies in the row or beyond its end.  Else the
// row's first and last vector may lie partly outside it; the thread that has one (`edge`) zeroes that part in a
// branch of its own, once for all units (a branch or a mask for each unit cost all threads more).
template <int VEC, int E, bool WHOLE>
struct Units {
    static constexpr int U = VEC > 1 ? E / VEC : E / 2;
    static constexpr int H = VEC > 1 ? VEC / 2 : 1;
    static constexpr int NV = E / VEC;
    int t, g, off, cols;  // thread of its group of g
    bool edge = false;    // a unit lies partly in the row
    __device__ __forceinline__ Units(int t, int g, int off, int cols) : t(t), g(g), off(off), cols(cols)
    {
        if constexpr (!WHOLE)
#pragma unroll
            for (int u = 0; u < U; ++u) edge |= !none(u) && !whole(u);
    }
    // column of element i of unit u: below 0 or past the end outside the row
    __device__ __forceinline__ int col(int u, int i) const { return VEC > 1 ? (u * g + t) * VEC + i - off : (2 * u + i) * g + t; }
    __device__ __forceinline__ bool in(int u, int i) const
    {
        return WHOLE ? col(u, 0) < cols : static_cast<unsigned>(col(u, i)) < static_cast<unsigned>(cols);
    }
    __device__ __forceinline__ bool none(int u) const { return col(u, 0) >= cols; }
    __device__ __forceinline__ bool whole(int u) const { return WHOLE || (VEC > 1 ? col(u, 0) >= 0 && col(u, 2 * H - 1) < cols : in(u, 1)); }
    // Zeroes the part of a partial unit that lies outside the row.
    __device__ __forceinline__ void cut(float2 (&d)[U][H]) const
    {
        if constexpr (!WHOLE) {
            if (edge) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (!none(u) && !whole(u)) {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            if (!in(u, 2 * i)) d[u][i].x = 0.f;
                            if (!in(u, 2 * i + 1)) d[u][i].y = 0.f;
                        }
                    }
            }
        }
    }
    // Whether some of the warp's elements may lie outside the row (all lanes of a warp ask).
    __device__ __forceinline__ bool ragged() const { return !WHOLE || __any_sync(0xffffffffu, none(U - 1)); }
    // Sets what lies outside the row to `value`.
    __device__ __forceinline__ void fill(float2 (&d)[U][H], float value) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (!in(u, 2 * i)) d[u][i].x = value;
                if (!in(u, 2 * i + 1)) d[u][i].y = value;
            }
    }
    template <typename T>
    __device__ __forceinline__ void widen(float2 (&d)[H], const Pack<T, VEC>& v) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) d[i] = make_float2(v.v[2 * i], v.v[2 * i + 1]);
        }
    }
    // The unit's values, beyond the row's end zero or, of single elements, `other` (before its beginning the row before, see cut).
    template <typename T, typename R>
    __device__ __forceinline__ void take(float2 (&d)[H], const R& ring, int slot, const T* row, int u, bool live, float other = 0.f) const
    {
        if constexpr (VEC == 1) {
            d[0] = make_float2(live && in(u, 0) ? mx::to_float(row[col(u, 0)]) : other, live && in(u, 1) ? mx::to_float(row[col(u, 1)]) : other);
        } else {
            Pack<T, VEC> v;
            ring.get(v, slot, u);
            widen(d, v);
        }
    }
    // The same where the row begins `shift` elements behind the ring's first vector but columns begin with the row: a
    // vector's values lie in two of the ring's, the second another thread's (of the last vector of all nothing lies there).
    template <typename T, typename R>
    __device__ __forceinline__ void take_shifted(float2 (&d)[H], const R& ring, int slot, int u, int shift) const
    {
        static_assert(sizeof(T) * VEC == 16, "a vector to a copy");
        const uint8_t* at = ring.at(slot, u, 0);
        const uint4 lo = *reinterpret_cast<const uint4*>(at);
        uint4 hi = make_uint4(0, 0, 0, 0);
        if (t + 1 < g)
            hi = *reinterpret_cast<const uint4*>(at + 16);
        else if (u + 1 < U)
            hi = *reinterpret_cast<const uint4*>(ring.at(slot, u + 1, 0) - (g - 1) * 16);
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        constexpr int PER = 4 / sizeof(T);  // elements of a word
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = shift & (2 * PER) ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = shift & PER ? w[i + 1] : w[i];
        Pack<T, VEC> v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint32_t*>(&v)[i] = PER == 2 ? __funnelshift_r(w[i], w[i + 1], 16 * (shift & 1)) : w[i];
        widen(d, v);
    }
    // Stores the values that lie in the row.  A vector is made before anything is asked, so that its store is one predicated
    // instruction (a branch around both cost the backward pass a quarter of its time), and a row's first and last vector wait for one branch at the end.
    template <typename T>
    __device__ __forceinline__ void put(T* row, const float2 (&d)[U][H], bool live) const
    {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Pack<T, VEC> o;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if constexpr (sizeof(T) == 2) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(d[u][i].x, d[u][i].y);
                        o.v[2 * i] = b.x;
                        o.v[2 * i + 1] = b.y;
                    } else {
                        o.v[2 * i] = d[u][i].x;
                        o.v[2 * i + 1] = d[u][i].y;
                    }
                }
                if (live && !none(u) && whole(u)) *reinterpret_cast<Pack<T, VEC>*>(row + col(u, 0)) = o;
            }
            if constexpr (WHOLE) return;
        }
        if (live && (VEC == 1 || edge)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (VEC == 1 || (!none(u) && !whole(u))) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        if (in(u, 2 * i)) mx::from_float(row[col(u, 2 * i)], d[u][i].x);
                        if (in(u, 2 * i + 1)) mx::from_float(row[col(u, 2 * i + 1)], d[u][i].y);
                    }
                }
        }
    }
    // The unit's values of a per-column fp32 vector: `other` where there is none, 0 outside the row.
    __device__ __forceinline__ void params(float2 (&d)[H], const float* v, int u, float other) const
    {
#pragma unroll
        for (int i = 0; i < H; ++i)
            d[i] = make_float2(!in(u, 2 * i) ? 0.f : v ? __ldg(v + col(u, 2 * i)) : other,
                               !in(u, 2 * i + 1) ? 0.f : v ? __ldg(v + col(u, 2 * i + 1)) : other);
    }
};

// Sums over the threads of a row; `buf` is a buffer that no thread reads any more.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[32])
{
#pragma unroll
    for (int o = (G ? G : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (G == 0) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
        __syncthreads();
        const bool have = (lane & 15) < static_cast<int>(blockDim.x >> 5);  // at most 16 warps, summed by each half of a warp
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = have ? buf[i][lane & 15] : 0.f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// Stores one vector's values as part of a quantised row (all lanes of a warp take part): the 32/VEC lanes that hold a
// block of 32 share its scale.  `data` is the row's, `scales` the row's first four bytes in the row's tiles; elements are stored for
// blocks below `live`, scale bytes for the first `tiles` scale tiles.
template <int VEC>
__device__ __forceinline__ void store_mx(const float2 (&v)[(VEC + 1) / 2], int col, uint8_t* data, uint8_t* scales, int live, int tiles)
{
    constexpr int LANES = mx::BLOCK / VEC;
    const int lane = threadIdx.x & 31;
    float largest = fabsf(v[0].x);
    if constexpr (VEC > 1)
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) largest = mx::max_abs3(largest, v[i].x, v[i].y);
    uint32_t m = mx::abs_bits(largest);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t byte = mx::scale_byte(m);
    const float inv = mx::inverse_scale(byte);
    const int b = col / mx::BLOCK;
    const bool in_data = b < live, in_tile = b < tiles * mx::TILE_BLOCKS;
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = VEC == 1 ? make_float2(i ? 0.f : v[0].x * inv, 0.f) : 2 * i < VEC ? mul2(v[i < VEC / 2 ? i : 0], make_float2(inv, inv)) : make_float2(0.f, 0.f);
        q[2 * i] = s.x;
        q[2 * i + 1] = s.y;
    }
    uint32_t word = mx::pack_e2m1x8(q);
    if constexpr (VEC == 8) {
        if (in_data) *reinterpret_cast<uint32_t*>(data + col / 2) = word;
    } else if constexpr (VEC == 4) {
        if (in_data) *reinterpret_cast<uint16_t*>(data + col / 2) = static_cast<uint16_t>(word);
    } else {  // one element to a lane: eight lanes' codes make a word
        word |= __shfl_xor_sync(0xffffffffu, word, 1) << 4;  // right in even lanes
        word |= __shfl_xor_sync(0xffffffffu, word, 2) << 8;
        word |= __shfl_xor_sync(0xffffffffu, word, 4) << 16;
        if (in_data && lane % 8 == 0) *reinterpret_cast<uint32_t*>(data + col / 2) = word;
    }
    if (in_tile && lane % LANES == 0) scales[b / 4 * mx::TILE_BYTES + (b & 3)] = static_cast<uint8_t>(byte);
}

// Forward.  TY = void: the result quantised; rows from p.rows to p.padded_rows are the scale tiles' padding.  The format's blocks
// begin with the row, so `off` is 0 there, and vectors of rows that do not start at 16 bytes are put together from the ring's,
// which takes one barrier more to a row (16384 x 2047 bf16: 45 us; element by element 190).
template <typename TX, typename TY, int VEC, int E, int G, int MOST, bool WHOLE>
__global__ void __launch_bounds__(MOST, FWD_RESIDENT<G, E, MOST>) fwd_rows(const TX* __restrict__ x, TY* y, const FwdParams p)
{
    constexpr bool MX = std::is_same_v<TY, void>;
    constexpr int ROWS = G ? MOST / G : 1, DEPTH = ring_depth(RowShape{G ? G : MOST, E, MOST}, sizeof(TX), 0);
    static_assert(!MX || G == 0 || (G * VEC >= mx::BLOCK && G * E >= mx::BLOCK * mx::TILE_BLOCKS), "a block's lanes lie in one group, which covers whole scale tiles");
    using Un = Units<VEC, E, WHOLE>;
    constexpr int U = Un::U, H = Un::H;
    extern __shared__ __align__(16) uint8_t ring_mem[];
    __shared__ float sums[2][1][32];
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int64_t end = MX ? p.padded_rows : p.rows;
    // rows of a warp run together, so that shuffles have all lanes
    const int g = G ? G : blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + (G ? threadIdx.x / (G ? G : 1) : 0);
    const int64_t lead = G && G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / (G ? G : 1) : first;
    constexpr bool SHIFTED = MX && VEC > 1 && !WHOLE;
    const int before = WHOLE || VEC == 1 ? 0 : static_cast<int>(first * p.x_stride % VEC);  // elements in front of a row
    const Un un(G ? threadIdx.x % (G ? G : 1) : threadIdx.x, g, SHIFTED ? 0 : before, p.cols);
    const int blocks = MX ? mx::cdiv(p.cols, mx::BLOCK) : 0, btiles = MX ? mx::cdiv(blocks, mx::TILE_BLOCKS) : 0;

    // The quantised norm alone has its ring know of whole rows (fp32 16384 x 4096 76 us, 84 without; but the gradient of 32768 x 4096 bf16
    // 163 us, 141 without).
    const Ring<TX, VEC == 1 ? 8 : VEC, VEC == 1 ? 1 : Un::NV, DEPTH, MX && WHOLE> ring(ring_mem, blockDim.x);
    auto ask = [&](int slot, int64_t r) {
        if constexpr (VEC > 1) {
            const int front = r < p.rows ? before : 0;
            ring.ask(slot, x + (r < p.rows ? r * p.x_stride : 0), un.t * VEC - front, g * VEC, r < p.rows ? p.cols : 0, front);
            ptx::cp_async_commit();
        }
    };
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) ask(k, first + k * step);

    float2 w[U][H], b[U][H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        un.params(w[u], p.weight, u, 1.f);
        un.params(b[u], p.bias, u, 0.f);
    }
    int slot = 0;
    for (int64_t r = first, r_lead = lead; r_lead < end; r += step, r_lead += step) {
        const bool live = r < p.rows;
        if constexpr (VEC > 1) ptx::cp_async_wait<DEPTH - 1>();
        float2 d[U][H];
        float2 s2 = make_float2(0.f, 0.f);
        if constexpr (SHIFTED) G ? __syncwarp() : __syncthreads();  // the others' copies have landed as well
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (SHIFTED)
                un.template take_shifted<TX>(d[u], ring, slot, u, before);
            else
                un.take(d[u], ring, slot, x + r * p.x_stride, u, live);
        }
        un.cut(d);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) s2 = add2(s2, d[u][i]);
        float s[1] = {s2.x + s2.y};
        row_sum<G>(s, sums[0]);
        if constexpr (SHIFTED && G) __syncwarp();  // (a block's threads met in the sum)
        ask(slot, r + DEPTH * step);  // what the slot held is in registers
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
        const float mean = s[0] * p.inv_cols;
        const float2 minus = make_float2(-mean, -mean);
        s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float2 m = un.none(u) ? make_float2(0.f, 0.f) : minus;  // zeros beyond the row stay
#pragma unroll
            for (int i = 0; i < H; ++i) d[u][i] = add2(d[u][i], m);
        }
        un.cut(d);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) s2 = fma2(d[u][i], d[u][i], s2);
        s[0] = s2.x + s2.y;
        row_sum<G>(s, sums[1]);
        const float rstd = rsqrtf(s[0] * p.inv_cols + p.eps);
        if (live && un.t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
        const float2 scale = make_float2(rstd, rstd);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < H; ++i) d[u][i] = fma2(mul2(d[u][i], scale), w[u][i], b[u][i]);
        // Outside the row lie zeros, of weight and bias too, but a NaN or infinite rstd makes NaN of them.  Asked of the whole warp, as a branch
        // that lanes may take apart costs the quantised norm 10% (401408 x 64 fp32: 58 us, 64 that way).
        if constexpr (MX)
            if (__any_sync(0xffffffffu, !(rstd <= FLT_MAX))) un.fill(d, 0.f);
        if constexpr (!MX) {
            un.put(y + r * p.y_stride, d, live);
        } else {
            uint8_t* data = p.data + r * (static_cast<int64_t>(blocks) * 16);
            uint8_t* scales = p.scales + mx::scale_at(r, 0, btiles);
            const int live_blocks = live ? blocks : 0, tiles = r < end ? btiles : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!live) {  // outside the row weight and bias are zero
#pragma unroll
                    for (int i = 0; i < H; ++i) d[u][i] = make_float2(0.f, 0.f);
                }
                if constexpr (VEC == 1) {
                    const float2 second[1] = {make_float2(d[u][0].y, 0.f)};
                    store_mx<1>(d[u], un.col(u, 0), data, scales, live_blocks, tiles);
                    store_mx<1>(second, un.col(u, 1), data, scales, live_blocks, tiles);
                } else {
                    store_mx<VEC>(d[u], un.col(u, 0), data, scales, live_blocks, tiles);
                }
            }
        }
    }
    if constexpr (VEC > 1) ptx::cp_async_wait_all();
}

// Backward: dx and, with SUMS, this block's part of dweight and dbias.
template <typename TX, typename TY, int VEC, int E, int G, int MOST, bool SUMS, bool WHOLE>
__global__ void __launch_bounds__(MOST, BWD_RESIDENT<G, E, MOST>) bwd_rows(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                                                  TX* __restrict__ dx, const BwdParams p)
{
    constexpr int ROWS = G ? MOST / G : 1, DEPTH = ring_depth(RowShape{G ? G : MOST, E, MOST}, sizeof(TX), sizeof(TY));
    using Un = Units<VEC, E, WHOLE>;
    constexpr int U = Un::U, H = Un::H;
    extern __shared__ __align__(16) uint8_t ring_mem[];
    __shared__ float sums[2][2][32];
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const int group = G ? G : blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + (G ? threadIdx.x / (G ? G : 1) : 0);
    const int64_t lead = G && G < 32 ? static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x & ~31) / (G ? G : 1) : first;
    const Un un(G ? threadIdx.x % (G ? G : 1) : threadIdx.x, group, WHOLE || VEC == 1 ? 0 : static_cast<int>(first * p.x_stride % VEC), p.cols);

    using RingX = Ring<TX, VEC == 1 ? 8 : VEC, VEC == 1 ? 1 : Un::NV, DEPTH, false>;
    using RingG = Ring<TY, VEC == 1 ? 8 : VEC, VEC == 1 ? 1 : Un::NV, DEPTH, false>;
    const RingX ring_x(ring_mem, blockDim.x);
    const RingG ring_g(ring_mem + RingX::THREAD_BYTES * blockDim.x, blockDim.x);
    auto ask = [&](int slot, int64_t r) {
        if constexpr (VEC > 1) {
            const bool live = r < p.rows;
            const int front = live ? un.off : 0;
            ring_x.ask(slot, x + (live ? r * p.x_stride : 0), un.t * VEC - front, group * VEC, live ? p.cols : 0, front);
            ring_g.ask(slot, dy + (live ? r * p.dy_stride : 0), un.t * VEC - front, group * VEC, live ? p.cols : 0, front);
            ptx::cp_async_commit();
        }
    };
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) ask(k, first + k * step);
    float mean = first < p.rows ? __ldg(p.mean + first) : 0.f, rstd = first < p.rows ? __ldg(p.rstd + first) : 0.f;

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
        const float2 minus = make_float2(-mean, -mean), scale = make_float2(rstd, rstd);
        mean = r + step < p.rows ? __ldg(p.mean + r + step) : 0.f;
        rstd = r + step < p.rows ? __ldg(p.rstd + r + step) : 0.f;
        if constexpr (VEC > 1) ptx::cp_async_wait<DEPTH - 1>();
        float2 xh[U][H], g[U][H];
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            un.take(xh[u], ring_x, slot, x + r * p.x_stride, u, live, -minus.x);
            un.take(g[u], ring_g, slot, dy + r * p.dy_stride, u, live);
        }
        // Outside the row dy is zero, but a normalised zero may be past fp32 where the row's values are not: there the mean stands in x's
        // place, of single elements always, else in the rows where that is so.  Warps that have nothing there do not ask (65536 x 1024
        // bf16 76.8 us, 80 where they do; fp32 16384 x 8191, single elements, 322 us, 374 with the question).
        if constexpr (VEC > 1) {
            un.cut(xh);
            un.cut(g);
            if (ragged && __any_sync(0xffffffffu, !(fabsf(minus.x * scale.x) <= FLT_MAX))) un.fill(xh, -minus.x);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                xh[u][i] = mul2(add2(xh[u][i], minus), scale);
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
            for (int i = 0; i < H; ++i) xh[u][i] = mul2(scale, fma2(xh[u][i], s1, add2(g[u][i], s0)));
        un.put(dx + r * p.cols, xh, live);
    }
    if constexpr (VEC > 1) ptx::cp_async_wait_all();
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
        float* mine = join + threadIdx.x / (G ? G : 1) * W;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = col(i);
            if (static_cast<unsigned>(c) < static_cast<unsigned>(p.cols)) {
                mine[c] = at_w(i);
                mine[ROWS * W + c] = at_b(i);
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
