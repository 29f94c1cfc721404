// One direction through the adapters, in [rows][from] -> mid [rows][rank] -> out [rows][to], by tiles of up to 128 rows of one adapter:
//
//   mid = scale * in w1^T,  out = act(base + mid w2^T)
//
// Forward w1 is a[e] and w2 is b[e], both K-major operands; backward (TRANS) w1 is b[e]^T and w2 a[e]^T, both MN-major.
//
// in, base and out each pass once over HBM and bind it: with rank r the matrix units have 2r flops to some 4 bytes.  A cluster
// of S CTAs shares a tile: each takes a part of `from` for the first product, 128/S rows of the join and a part of `to` for the
// second.  Two CTAs stay on an SM up to rank 64, each at a phase of its own.  mid never leaves the chip but for the copy that the gradients need.
//
// First product: rows of `in` are gathered by the plan's order with cp.async, 128 bytes of a row at a time, 128 x rank x 64 a stage.  The sums over
// the parts meet in shared memory as fp32, are joined in the CTAs' order and cut into three bf16 parts that
// hold all 24 bits: the second product, K = 3 * rank, is that of an fp32 mid.
//
// Second product: mid's parts are its A operand in tensor memory (from shared memory they would be read once for each chunk and take
// most of its bandwidth), 64 columns of `to` (128 of tiles of 64 rows) its B.  Two groups of 8 warps finish chunks by turns.  A thread reads the accumulator in the 16 x 256-bit layout, 2
// neighbouring columns of a lane in each group of 8; w2's rows are placed in shared memory in an order that makes these 8 neighbouring columns of out, so base and
// out move in 16-byte vectors straight between registers and memory, base a chunk ahead.
//
// Every wait is bounded: on running out the status word is set and the CTA goes through its remaining barriers without waiting or storing.
#pragma once

#include "adapter_params.cuh"
#include "adapter_ptx.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

constexpr int P_WARPS = 16, P_LOADERS = 32 * P_WARPS, P_THREADS = P_LOADERS + 32;
constexpr int P_GROUP = P_LOADERS / 2;  // threads that finish a chunk
constexpr uint64_t P_WAIT_NS = 1000000000ull;
constexpr uint32_t P_TMEM = 512;  // the first product's sums, then 256 columns of chunks; mid's parts at the end

template <bool TRANS, bool VEC, int HALVED, typename TB, typename TO>
struct Pass {
    static constexpr int ROWS = TILE >> HALVED, COLS = 64 << HALVED;  // of a tile; of `to`, in a chunk
    static constexpr int BUFS = 4 >> HALVED;                           // accumulators of chunks
    static constexpr int LANES = 32 >> HALVED;                        // of a warp's 32 lanes of tensor memory that hold rows

    const PassParams& p;
    const PassSmem s;
    uint8_t* mem;
    uint64_t *full, *empty, *done, *w2_full, *d_full, *d_empty, *mid_full;
    int* ids;  // numbers of the tile's rows
    uint32_t* slot;
    volatile uint32_t* abort_flag;
    int tid, warp, lane, rank_in, e, n_stages, n_bufs;
    int group, gtid;  // of two that finish chunks by turns, and the thread of it

    Piece piece;

    __device__ __forceinline__ Pass(const PassParams& p, uint8_t* raw) : p(p), s(p.rank, HALVED), mem(raw)
    {
        n_stages = s.stages();
        n_bufs = s.chunks();
        full = reinterpret_cast<uint64_t*>(raw + s.area() + s.chunk());
        empty = full + P_MOST_STAGES;
        done = empty + P_MOST_STAGES;
        w2_full = done + 1;
        d_full = w2_full + P_MOST_CHUNKS;
        d_empty = d_full + 4;
        mid_full = d_empty + 4;
        ids = reinterpret_cast<int*>(mid_full + 1);
        slot = reinterpret_cast<uint32_t*>(ids + TILE);
        abort_flag = slot + 1;
        tid = threadIdx.x;
        warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, as the compiler then knows
        lane = tid & 31;
        rank_in = blockIdx.x % p.splits;
        group = warp >> 3;
        gtid = tid & (P_GROUP - 1);
    }
    // Once a wait has run out, `ok` is false and the thread waits no more: it goes on through its barriers with whatever is in memory.
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& ok) const
    {
        if (!ptx::mbar_try_wait(bar, parity) && ok && !ptx::mbar_wait(bar, parity, P_WAIT_NS)) {
            ok = false;
            *abort_flag = 1u;
        }
    }
    __device__ __forceinline__ float* mids() const { return reinterpret_cast<float*>(mem + s.area() - s.sums()); }
    __device__ __forceinline__ uint8_t* w2_buf(int i) const { return i ? mem + s.area() - s.sums() - i * s.chunk() : mem + s.area(); }

    // 16 bytes of row elements from `src`, `valid` elements of them; aligned copies run by themselves, others go through registers.
    __device__ __forceinline__ void copy8(uint32_t dst, const __nv_bfloat16* src, int valid) const
    {
        if constexpr (VEC) {
            ptx::cp_async_16s(dst, valid > 0 ? src : p.w1, valid > 0 ? 16 : 0);
        } else {
            uint32_t v[4] = {0u, 0u, 0u, 0u};
            if (valid > 0) mx::load_any<4, 2>(v, src, valid < 8 ? 2 * valid : 16);
            ptx::st_shared_v4(dst, v[0], v[1], v[2], v[3]);
        }
    }
    // This warp's part of what `bar` counts is there (its threads have waited for their copies).  One arrival to a warp: a barrier takes its
    // arrivals one after another, and 512 of them cost as much as the stage.
    __device__ __forceinline__ void arrive(uint64_t* bar) const
    {
        if (!VEC) ptx::fence_proxy_async_smem();
        __syncwarp();
        ptx::mbar_arrive_if(bar, lane == 0);
    }

    // The accumulator's lane of row i: a halved tile has 16 rows in each warp's 32 lanes, so that all warps finish chunks.
    __device__ __forceinline__ static int lane_of(int i) { return HALVED ? (i >> 4) * 32 + (i & 15) : i; }

    // Where a loader's copies of an MN-major w1 or a K-major w2 go: 64 rows of rank/8 16-byte columns, one after another in memory.
    // (Addresses are kept in registers: computed for each copy they cost the loaders more time than the copies.)
    static constexpr int PLACES = 64 * MOST_RANK / 8 / (TRANS ? P_LOADERS : P_GROUP);
    uint32_t place[PLACES];
    __device__ __forceinline__ void make_places()
    {
        const int per = p.rank >> 3;
#pragma unroll
        for (int j = 0; j < PLACES; ++j) {
            const int i = TRANS ? tid + P_LOADERS * j : gtid + P_GROUP * j, row = i / per, c8 = i - row * per;
            const int n = (row & 32) + 8 * ((row >> 1) & 3) + 2 * ((row >> 3) & 3) + (row & 1);  // of w2, as below
            place[j] = row >= 64 ? 0xffffffffu : TRANS ? (row & 7) * 16 + (row >> 3) * 128 + c8 * W1_COLUMN : (n & 7) * 16 + (n >> 3) * 144 + c8 * s.column();
        }
    }

    // Columns f0 .. f0+63 of the tile's rows and of w1.  rows: at this thread's 16-byte column of every 64th row.
    __device__ __forceinline__ void load_stage(uint8_t* st, int f0, const __nv_bfloat16* const (&rows)[ROWS / 64]) const
    {
        const uint32_t at = ptx::smem_addr(st), w_at = at + TILE * P_STEP * 2;
        const int64_t size = static_cast<int64_t>(p.rank) * p.from;
        const __nv_bfloat16* w = p.w1 + e * size;
        const int row = tid >> 3, c8 = tid & 7, l = lane_of(row);
        const uint32_t swizzled = (c8 ^ (row & 7)) << 4, mine = l * 128 + swizzled;  // 128-byte swizzle
        if (VEC && f0 + P_STEP <= p.from) {
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i)
                ptx::cp_async_16_if(at + mine + 8192 * i, rows[i] + f0, row + 64 * i < piece.rows);
            if constexpr (!TRANS) {
                const __nv_bfloat16* src = w + static_cast<int64_t>(row) * p.from + f0 + 8 * c8;
                ptx::cp_async_16_if(w_at + row * 128 + swizzled, src, row < p.rank);
                ptx::cp_async_16_if(w_at + row * 128 + swizzled + 8192, src + 64 * static_cast<int64_t>(p.from), row + 64 < p.rank);
            } else {
                const __nv_bfloat16* src = w + static_cast<int64_t>(f0) * p.rank + 8 * tid;
#pragma unroll
                for (int i = 0; i < PLACES; ++i)
                    ptx::cp_async_16_if(w_at + place[i], src + 8 * P_LOADERS * i, place[i] != 0xffffffffu);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < ROWS / 64; ++i)
            if (row + 64 * i < piece.rows) copy8(at + mine + 8192 * i, rows[i] + f0, p.from - f0 - 8 * c8);
        if constexpr (!TRANS) {
            for (int r = row; r < p.rank; r += 64)
                copy8(w_at + r * 128 + swizzled, w + static_cast<int64_t>(r) * p.from + f0 + 8 * c8, p.from - f0 - 8 * c8);
        } else {
            for (int i = tid; i < s.rp * 8; i += P_LOADERS) {  // 64 rows of rp/8 16-byte columns
                const int k = (i >> 1) & 63, n8 = 2 * (i >> 7) + (i & 1);
                const int left = f0 + k < p.from ? p.rank - 8 * n8 : 0;
                copy8(w_at + (k & 7) * 16 + n8 * W1_COLUMN + (k >> 3) * 128, w + static_cast<int64_t>(f0 + k) * p.rank + 8 * n8, left);
            }
        }
    }

    // w2's columns of a chunk from c0 on, by a group: column c of 32 becomes row 8((c>>1)&3) + 2(c>>3) + (c&1) of the operand.
    __device__ __forceinline__ void load_w2(uint8_t* buf, int c0) const
    {
        const int64_t size = static_cast<int64_t>(p.rank) * p.to;
        const __nv_bfloat16* w = p.w2 + e * size;
        uint32_t at = ptx::smem_addr(buf);
#pragma unroll
        for (int half = 0; half < COLS / 64; ++half, at += 8 * 144, c0 += 64) {
            if (VEC && c0 + 64 <= p.to) {
                if constexpr (!TRANS) {
                    const __nv_bfloat16* src = w + static_cast<int64_t>(c0) * p.rank + 8 * gtid;
#pragma unroll
                    for (int i = 0; i < PLACES; ++i)
                        ptx::cp_async_16_if(at + place[i], src + 8 * P_GROUP * i, place[i] != 0xffffffffu);
                } else {
                    const int c = 2 * lane, gwarp = warp & 7;
                    uint32_t dst = at + gwarp * 16 + ((c >> 3) & 3) * 4 + (((c >> 1) & 3) + 4 * (c >> 5)) * 144;
                    const __nv_bfloat16* src = w + static_cast<int64_t>(gwarp) * p.to + c0 + c;
                    for (int k = gwarp; k < s.rp; k += 16, dst += 2 * s.column(), src += 16 * static_cast<int64_t>(p.to)) {
                        ptx::cp_async_4_if(dst, src, k < p.rank);
                        ptx::cp_async_4_if(dst + s.column(), src + 8 * static_cast<int64_t>(p.to), k + 8 < p.rank);
                    }
                }
            } else if constexpr (!TRANS) {
                for (int i = gtid; i < s.rp * 8; i += P_GROUP) {
                    const int n = (i >> 1) & 63, k8 = 2 * (i >> 7) + (i & 1);
                    const int c = c0 + (n & 32) + 8 * ((n >> 1) & 3) + 2 * ((n >> 3) & 3) + (n & 1);
                    copy8(at + (n & 7) * 16 + (n >> 3) * 144 + k8 * s.column(), w + static_cast<int64_t>(c) * p.rank + 8 * k8, c < p.to ? p.rank - 8 * k8 : 0);
                }
            } else {
                for (int i = gtid; i < s.rp * 32; i += P_GROUP) {
                    const int k = i >> 5, c = 2 * (i & 31);
                    const uint32_t dst = at + (k & 7) * 16 + ((c >> 3) & 3) * 4 + (((c >> 1) & 3) + 4 * (c >> 5)) * 144 + (k >> 3) * s.column();
                    const __nv_bfloat16* src = w + static_cast<int64_t>(k) * p.to + c0 + c;
                    const int left = k < p.rank ? p.to - c0 - c : 0;
                    if constexpr (VEC) {
                        ptx::cp_async_4(dst, left > 0 ? src : p.w1, left > 0 ? 4 : 0);
                    } else {
                        const uint32_t lo = left > 0 ? __bfloat16_as_ushort(__ldg(src)) : 0u, hi = left > 1 ? __bfloat16_as_ushort(__ldg(src + 1)) : 0u;
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(lo | hi << 16) : "memory");
                    }
                }
            }
        }
    }
    // The part of a chunk of w2 that pads an odd number of 8 ranks; whole copies do not reach it.
    __device__ __forceinline__ void clear_pad(uint8_t* buf) const
    {
        if (!VEC || !(p.rank & 8)) return;
        if (gtid < COLS) ptx::st_shared_v4(ptx::smem_addr(buf) + (gtid & 7) * 16 + (gtid >> 3) * 144 + (p.rank >> 3) * s.column(), 0u, 0u, 0u, 0u);
        ptx::fence_proxy_async_smem();
    }

    // This CTA's rows of the sums over the cluster: scaled, to mid, and on to every CTA.
    template <int S>
    __device__ __forceinline__ void join(const float* sums, float scale) const
    {
        constexpr int SHARE = ROWS / S;
        const int eighths = s.rp >> 3;
        for (int i = tid; i < SHARE * eighths; i += P_THREADS) {  // neighbouring lanes read neighbouring parts of a row
            const int own = i / eighths, row = rank_in * SHARE + own, r = 8 * (i - own * eighths);
            const float* at = sums + row * s.pitch() + r;
            float v[8] = {};
            if (row < piece.rows) {
                float4 u[S][2];
#pragma unroll
                for (int k = 0; k < S; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (S == 1)
                            u[k][h] = reinterpret_cast<const float4*>(at)[h];
                        else
                            u[k][h] = ptx::ld_cluster_v4(ptx::mapa_shared(ptx::smem_addr(at + 4 * h), k));
                    }
#pragma unroll
                for (int k = 0; k < S; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        v[4 * h] += u[k][h].x;
                        v[4 * h + 1] += u[k][h].y;
                        v[4 * h + 2] += u[k][h].z;
                        v[4 * h + 3] += u[k][h].w;
                    }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r + j < p.rank ? v[j] * scale : 0.f;
                if (p.mid) {
                    float* mid = p.mid + static_cast<int64_t>(ids[row]) * p.rank + r;
                    if (VEC && r < p.rank) {
                        reinterpret_cast<float4*>(mid)[0] = make_float4(v[0], v[1], v[2], v[3]);
                        reinterpret_cast<float4*>(mid)[1] = make_float4(v[4], v[5], v[6], v[7]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (r + j < p.rank) mid[j] = v[j];
                    }
                }
            }
            float* mine = mids() + row * s.pitch() + r;
            reinterpret_cast<float4*>(mine)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(mine)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        ptx::fence_proxy_async_smem();
        __syncthreads();
        if (S > 1 && tid < S && tid != rank_in) {
            const uint32_t at = ptx::smem_addr(mids() + rank_in * SHARE * s.pitch());
            ptx::bulk_to_cluster(ptx::mapa_shared(at, tid), at, SHARE * s.pitch() * 4, ptx::mapa_shared(ptx::smem_addr(mid_full), tid));
        }
    }

    // mid's three parts to tensor memory, two neighbouring ranks to a column.
    __device__ __forceinline__ void store_parts(uint32_t to) const
    {
        const float* row = mids() + (LANES * (warp & 3) + (lane & (LANES - 1))) * s.pitch();
        for (int r = 16 * (warp >> 2); r < s.rp; r += 64) {
            uint32_t part[3][8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float4 v = *reinterpret_cast<const float4*>(row + r + 2 * j);
                uint32_t a[3], b[3], c[3], d[3];
                split3(v.x, a[0], a[1], a[2]);
                split3(v.y, b[0], b[1], b[2]);
                split3(v.z, c[0], c[1], c[2]);
                split3(v.w, d[0], d[1], d[2]);
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    part[q][j] = a[q] | b[q] << 16;
                    part[q][j + 1] = c[q] | d[q] << 16;
                }
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) ptx::tmem_st_32x32b_x8(to + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + ((q * s.rp + r) >> 1), part[q]);
        }
        ptx::tmem_st_wait();
    }

    // A thread finishes four times 8 neighbouring elements of a chunk, SIDES side by side at 32 columns' distance in each of 4 / SIDES rows, 8 rows
    // apart.  It holds HOLD of them at a time: 64 bytes of base.
    static constexpr int SIDES = 1 << HALVED;
    static constexpr int HOLD = sizeof(TB) == 2 ? 4 : 2, TURNS = 4 / HOLD, WORDS = 2 * sizeof(TB);
    struct Held {
        uint32_t u[HOLD][WORDS];
    };
    const TB* base_at[4 / SIDES];
    TO* out_at[4 / SIDES];
    __device__ __forceinline__ static constexpr int row_index(int i) { return HALVED ? i & 1 : i; }
    __device__ __forceinline__ static constexpr int side_of(int i) { return HALVED ? i >> 1 : 0; }
    __device__ __forceinline__ int row_of(int i) const { return LANES * (warp & 3) + (lane >> 2) + 8 * row_index(i); }
    __device__ __forceinline__ int col_of(int i, int c0) const { return c0 + 32 * SIDES * ((warp >> 2) & 1) + 32 * side_of(i) + 8 * (lane & 3); }
    __device__ __forceinline__ void make_rows()
    {
#pragma unroll
        for (int i = 0; i < 4 / SIDES; ++i) {
            const int64_t t = ids[row_of(i)];
            row_here[i] = row_of(i) < piece.rows;
            base_here[i] = row_here[i] && p.base;
            base_at[i] = static_cast<const TB*>(p.base) + t * p.base_stride + col_of(i, 0);
            out_at[i] = static_cast<TO*>(p.out) + t * p.out_stride + col_of(i, 0);
        }
    }
    bool row_here[4 / SIDES], base_here[4 / SIDES];  // the thread's rows are of the tile; and there is a base
    // Turn `turn` of the chunk at c0; `whole`: all its columns exist.
    __device__ __forceinline__ void load_base(Held& b, int turn, int c0, bool whole, bool wanted = true) const
    {
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i = turn * HOLD + k;
            const TB* src = base_at[row_index(i)] + c0 + 32 * side_of(i);
            if constexpr (VEC) {
#pragma unroll
                for (int j = 0; j < WORDS; j += 4) {
                    const uint4 q = ptx::ld_stream_v4_if(reinterpret_cast<const uint4*>(src) + j / 4, wanted && base_here[row_index(i)] && (whole || col_of(i, c0) < p.to));
                    b.u[k][j] = q.x, b.u[k][j + 1] = q.y, b.u[k][j + 2] = q.z, b.u[k][j + 3] = q.w;
                }
            } else {
                const int left = wanted && base_here[row_index(i)] ? p.to - col_of(i, c0) : 0;
                TB* v = reinterpret_cast<TB*>(b.u[k]);
#pragma unroll
                for (int j = 0; j < WORDS; ++j) b.u[k][j] = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) v[j] = src[j];
            }
        }
    }
    // out = act(base + sum) for a turn: `v` the chunk's sums as they come from tensor memory.
    __device__ __forceinline__ void finish(const Held& b, const uint32_t (&v)[2][16], int turn, int c0, bool whole, bool live) const
    {
        float2 f[HOLD][4];
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i = turn * HOLD + k;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 sum = make_float2(__uint_as_float(v[i >> 1][4 * j + 2 * (i & 1)]), __uint_as_float(v[i >> 1][4 * j + 2 * (i & 1) + 1]));
                const float2 base = sizeof(TB) == 2 ? make_float2(__uint_as_float(b.u[k][j] << 16), __uint_as_float(b.u[k][j] & 0xffff0000u))
                                                    : make_float2(__uint_as_float(b.u[k][2 * j % WORDS]), __uint_as_float(b.u[k][(2 * j + 1) % WORDS]));
                f[k][j] = mx::add2(sum, base);
            }
        }
        if (p.relu)
#pragma unroll
            for (int k = 0; k < HOLD; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[k][j] = make_float2(__uint_as_float(ptx::relu_nan(__float_as_uint(f[k][j].x))), __uint_as_float(ptx::relu_nan(__float_as_uint(f[k][j].y))));
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i = turn * HOLD + k;
            TO* row = out_at[row_index(i)] + c0 + 32 * side_of(i);
            if constexpr (VEC) {
                const bool here = live && row_here[row_index(i)] && (whole || col_of(i, c0) < p.to);
                if constexpr (sizeof(TO) == 4) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        ptx::st_stream_v4_if(row + 4 * h, make_uint4(__float_as_uint(f[k][2 * h].x), __float_as_uint(f[k][2 * h].y), __float_as_uint(f[k][2 * h + 1].x),
                                                                     __float_as_uint(f[k][2 * h + 1].y)), here);
                } else {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(f[k][j].x, f[k][j].y);
                        o[j] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    ptx::st_stream_v4_if(row, make_uint4(o[0], o[1], o[2], o[3]), here);
                }
            } else {
                const int left = live && row_here[row_index(i)] ? p.to - col_of(i, c0) : 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) mx::from_float(row[j], j % 2 ? f[k][j / 2].y : f[k][j / 2].x);
            }
        }
    }

    // Base's first chunks to L2, where HBM works on them while the sums are joined.
    static constexpr int AHEAD = 4;
    __device__ __forceinline__ void prefetch_base(int chunk0, int chunk1) const
    {
        constexpr int LINES = AHEAD * COLS * sizeof(TB) / 128, EACH = 128 / sizeof(TB);
        if (!p.base || !p.out) return;
        for (int i = tid; i < piece.rows * LINES; i += P_LOADERS) {
            const int row = i / LINES, c = chunk0 * COLS + (i - row * LINES) * EACH;
            if (c < p.to && c < chunk1 * COLS) ptx::prefetch_l2(static_cast<const TB*>(p.base) + ids[row] * p.base_stride + c);
        }
    }

    // The first filling of w2's buffers i0 .. i1, each by the group whose chunk it is for, and the word that they are there.
    __device__ __forceinline__ void fill(int i0, int i1, int chunk0, int chunk1) const
    {
        for (int i = i0 + ((i0 ^ group) & 1); i < i1; i += 2) {
            clear_pad(w2_buf(i));
            if (chunk0 + i < chunk1) load_w2(w2_buf(i), (chunk0 + i) * COLS);
        }
        ptx::cp_async_commit();
    }
    __device__ __forceinline__ void filled(int i0, int i1) const
    {
        for (int i = i0 + ((i0 ^ group) & 1); i < i1; i += 2) arrive(&w2_full[i]);
    }

    // Rows without an adapter: out = act(base), mid = 0.
    __device__ __forceinline__ void without(int chunk0, int chunk1) const
    {
        if (p.mid && rank_in == 0)
            for (int i = tid; i < piece.rows * p.rank; i += P_THREADS)
                p.mid[static_cast<int64_t>(ids[i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (!p.out || warp >= P_WARPS) return;
        for (int c = chunk0 + group; c < chunk1; c += 2)
#pragma unroll
            for (int turn = 0; turn < TURNS; ++turn) {
                Held b;
                load_base(b, turn, c * COLS, false);
                const uint32_t none[2][16] = {};
                finish(b, none, turn, c * COLS, false, true);
            }
    }

    __device__ __forceinline__ void run()
    {
        if (tid == 0) {
            for (int i = 0; i < n_stages; ++i) {
                ptx::mbar_init(&full[i], P_WARPS);
                ptx::mbar_init(&empty[i], 1);
            }
            ptx::mbar_init(done, 1);
            for (int i = 0; i < n_bufs; ++i) ptx::mbar_init(&w2_full[i], P_WARPS / 2);
            for (int i = 0; i < BUFS; ++i) {
                ptx::mbar_init(&d_full[i], 1);
                ptx::mbar_init(&d_empty[i], P_WARPS / 2);
            }
            ptx::mbar_init(mid_full, 1);
            if (p.splits > 1) ptx::mbar_arrive_expect_tx(mid_full, (ROWS - ROWS / p.splits) * s.pitch() * 4);
            *abort_flag = 0u;
            ptx::mbar_init_fence();
        }
        if (warp == P_WARPS) {
            ptx::tmem_alloc(slot, P_TMEM);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        const uint32_t tmem = *slot;
        ptx::grid_dependency_wait();
        const int block = blockIdx.x / p.splits;
        piece = p.plan.tiles[block >> HALVED];  // the same for the whole cluster
        if constexpr (HALVED) {
            piece.first += (block & 1) * ROWS;
            piece.rows -= (block & 1) * ROWS;
            if (piece.rows > ROWS) piece.rows = ROWS;
        }
        e = piece.adapter;
        const int chunks = p.out ? (p.to + COLS - 1) / COLS : 0;
        const int chunk0 = static_cast<int>(static_cast<int64_t>(rank_in) * chunks / p.splits), chunk1 = static_cast<int>(static_cast<int64_t>(rank_in + 1) * chunks / p.splits);
        if (piece.rows > 0) {
            if (tid < TILE) ids[tid] = p.plan.order[piece.first + (tid < piece.rows ? tid : 0)];
            __syncthreads();
            if (warp < P_WARPS) make_rows();
            if (e < p.adapters)
                with(tmem, chunk0, chunk1);
            else
                without(chunk0, chunk1);
        }
        ptx::tc_fence_before();
        __syncthreads();
        if (warp == P_WARPS) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(tmem, P_TMEM);
        }
    }

    __device__ __forceinline__ void with(uint32_t tmem, int chunk0, int chunk1)
    {
        const int steps = (p.from + P_STEP - 1) / P_STEP;
        const int s0 = static_cast<int>(static_cast<int64_t>(rank_in) * steps / p.splits), s1 = static_cast<int>(static_cast<int64_t>(rank_in + 1) * steps / p.splits);
        bool ok = true;
        const float scale = p.scale ? __ldg(p.scale + e) : 1.f;
        if (warp < P_WARPS) {
            const __nv_bfloat16* rows[ROWS / 64];
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i) rows[i] = p.in + ids[(tid >> 3) + 64 * i] * p.in_stride + 8 * (tid & 7);
            if (VEC) make_places();
            constexpr int LAG = VEC ? 3 : 0;  // stages on their way behind the one that is asked for
            int at = 0, told = 0;
            uint32_t free_phase = 1u;
            for (int it = 0; it < s1 - s0; ++it) {
                wait(&empty[at], free_phase, ok);
                load_stage(mem + at * s.stage(), (s0 + it) * P_STEP, rows);
                at = at + 1 == n_stages ? 0 : at + 1;
                free_phase = at ? free_phase : free_phase ^ 1u;
                if (VEC) {
                    ptx::cp_async_commit();
                    ptx::cp_async_wait<LAG>();
                }
                if (it < LAG) continue;
                arrive(&full[told]);
                told = told + 1 == n_stages ? 0 : told + 1;
            }
            if (VEC) {
                ptx::cp_async_wait_all();
                for (int i = s1 - s0 < LAG ? s1 - s0 : LAG; i > 0; --i) {
                    arrive(&full[told]);
                    told = told + 1 == n_stages ? 0 : told + 1;
                }
            }
            prefetch_base(chunk0, chunk1);
            fill(0, 1, chunk0, chunk1);
        } else {
            int at = 0;
            uint32_t phase = 0u;
            for (int it = 0; it < s1 - s0; ++it) {
                wait(&full[at], phase, ok);
                __syncwarp();  // what follows is the whole warp's
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
                const uint32_t a = ptx::smem_addr(mem + at * s.stage()), b = a + TILE * P_STEP * 2;
                ptx::mma_bf16_elect_x4(tmem, ptx::sw128_kmajor_desc(a), TRANS ? ptx::plain_mnmajor_desc(b, 128, W1_COLUMN) : ptx::sw128_kmajor_desc(b),
                                       32 / 16, (TRANS ? 256 : 32) / 16, TRANS ? ptx::idesc_bf16_f32_bmn(TILE, s.rp) : ptx::idesc_bf16_f32(TILE, s.rp), it > 0);
                ptx::mma_commit_elect(&empty[at]);
                at = at + 1 == n_stages ? 0 : at + 1;
                phase = at ? phase : phase ^ 1u;
            }
            ptx::mma_commit_elect(done);
        }
        __syncwarp();
        wait(done, 0, ok);
        __syncwarp();
        // The ring is free: the sums, and w2's second chunk.
        float* sums = reinterpret_cast<float*>(mem);
        if (warp < P_WARPS) {
            ptx::tc_fence_after();
            const int row = LANES * (warp & 3) + lane;
            for (int c = 16 * (warp >> 2); c < s.rp; c += 64) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c, v);
                ptx::tmem_ld_wait();
                const uint32_t at = ptx::smem_addr(sums + row * s.pitch() + c);
                if (lane < LANES)
#pragma unroll
                    for (int i = 0; i < 4; ++i) ptx::st_shared_v4(at + 16 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                __syncwarp();
            }
            ptx::tc_fence_before();
        }
        if (p.splits > 1)
            ptx::cluster_sync();
        else
            __syncthreads();
        switch (p.splits) {
            case 1: join<1>(sums, scale); break;
            case 2: join<2>(sums, scale); break;
            case 4: join<4>(sums, scale); break;
            default: join<8>(sums, scale); break;
        }
        if (warp < P_WARPS) fill(1, s.early_chunks(), chunk0, chunk1);
        // All of mid is here: none of this CTA's peers reads its sums any more, and what they sent has come.
        if (p.splits > 1) {
            wait(mid_full, 0, ok);
            __syncwarp();
            ptx::cluster_arrive_relaxed();
        }
        const uint32_t parts = tmem + P_TMEM - 3 * s.rp / 2;
        if (warp < P_WARPS) {
            store_parts(parts);
            ptx::tc_fence_before();
        }
        __syncthreads();
        if (warp < P_WARPS) {
            ptx::cp_async_wait_all();
            filled(0, s.early_chunks());
            fill(s.early_chunks(), n_bufs, chunk0, chunk1);
        }
        const int n = chunk1 - chunk0;
        if (warp == P_WARPS) {
            ptx::tc_fence_after();
            int buf = 0;
            uint32_t phase = 0u;
            for (int j = 0; j < n; ++j) {
                const int b = j & (BUFS - 1);
                wait(&w2_full[buf], phase, ok);
                wait(&d_empty[b], (static_cast<uint32_t>(j / BUFS) & 1u) ^ 1u, ok);
                __syncwarp();
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
                const uint32_t w = ptx::smem_addr(w2_buf(buf));
                buf = buf + 1 == n_bufs ? 0 : buf + 1;
                phase = buf ? phase : phase ^ 1u;
                const uint64_t wd = ptx::plain_kmajor_desc(w, s.column(), 144), w_step = 2 * s.column() / 16;
                const uint32_t idesc = TRANS ? ptx::idesc_bf16_f32_bmn(TILE, COLS) : ptx::idesc_bf16_f32(TILE, COLS);
                const int whole = s.rp / 32;  // of the reduction, in twice three MMAs
                for (int k = 0; k < whole; ++k) ptx::mma_bf16_parts_x2(tmem + COLS * b, parts + 16 * k, wd + 2 * k * w_step, s.rp / 2, w_step, idesc, k > 0);
                if (s.rp & 16) ptx::mma_bf16_parts(tmem + COLS * b, parts + 16 * whole, wd + 2 * whole * w_step, s.rp / 2, idesc, whole > 0);
                ptx::mma_commit_elect(&d_full[b]);
            }
        } else if (group < n) {
            // This group's chunks, every other one; base a turn ahead, in two sets of registers by turns (a copy between them would wait for what
            // is on its way).
            Held held[2];
            load_base(held[0], 0, (chunk0 + group) * COLS, false);
            int buf = group % n_bufs, before = 0;  // w2's buffer of this chunk and of the group's last one
            for (int j0 = group; j0 < n; j0 += 4 / TURNS)
#pragma unroll
                for (int jj = 0; jj < 2 / TURNS; ++jj) {
                    const int j = j0 + 2 * jj;
                    if (j >= n) break;
                    const int b = j & (BUFS - 1), c0 = (chunk0 + j) * COLS;
                    const bool whole = c0 + COLS <= p.to, next = c0 + 3 * COLS <= p.to;
                    if (TURNS == 2)
                        load_base(held[1], 1, c0, whole);
                    else
                        load_base(held[(jj + 1) & 1], 0, c0 + 2 * COLS, next, j + 2 < n);
                    wait(&d_full[b], static_cast<uint32_t>(j / BUFS) & 1u, ok);
                    __syncwarp();
                    ptx::tc_fence_after();
                    uint32_t v[2][16];
                    const uint32_t at = tmem + COLS * b + 32 * SIDES * ((warp >> 2) & 1) + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
                    ptx::tmem_ld_16x256b_x4(at, v[0]);
                    ptx::tmem_ld_16x256b_x4(at + (HALVED ? 32u : 16u << 16), v[1]);
                    // w2 for this buffer's next chunk, and word of what was asked for a turn ago
                    if (j + n_bufs < n) load_w2(w2_buf(buf), c0 + n_bufs * COLS);
                    ptx::cp_async_commit();
                    ptx::cp_async_wait<1>();
                    if (j < 2)
                        filled(s.early_chunks(), n_bufs);
                    else if (j - 2 + n_bufs < n)
                        arrive(&w2_full[before]);
                    before = buf;
                    buf += 2;
                    buf = buf >= n_bufs ? buf - n_bufs : buf;
                    ptx::tmem_ld_wait();
                    ptx::tc_fence_before();
                    ptx::mbar_arrive_if(&d_empty[b], lane == 0);
                    finish(held[TURNS == 1 ? jj & 1 : 0], v, 0, c0, whole, ok);
                    if constexpr (TURNS == 2) {
                        load_base(held[0], 0, c0 + 2 * COLS, next, j + 2 < n);
                        finish(held[1], v, 1, c0, whole, ok);
                    }
                }
        }
        __syncwarp();
        ptx::cp_async_wait_all();
        if (!ok && lane == 0 && p.status) atomicMax(p.status, 6u);
        __syncwarp();
        if (p.splits > 1) ptx::cluster_wait();  // what this CTA sent has been received
    }
};

template <bool TRANS, bool VEC, int HALVED, typename TB, typename TO>
__global__ void __launch_bounds__(P_THREADS, 1) pass_tiles(const __grid_constant__ PassParams p)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    Pass<TRANS, VEC, HALVED, TB, TO> pass(p, raw);
    pass.run();
}

template <bool TRANS, bool VEC, int HALVED, typename TB, typename TO>
int start_pass_as(const PassParams& p, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const auto kernel = pass_tiles<TRANS, VEC, HALVED, TB, TO>;
    if (!mx::allow_smem(kernel, P_ROOM, done)) return CONV2D_ERR_CUDA;
    const int64_t grid = (static_cast<int64_t>(p.plan.n_tiles) << HALVED) * p.splits;
    if (grid > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    return mx::launch(kernel, grid, P_THREADS, P_ROOM, stream, p.splits, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

template <bool TRANS, bool VEC, int HALVED>
int start_pass_by_types(const PassParams& p, int32_t base, int32_t out, cudaStream_t stream)
{
    using B = __nv_bfloat16;
    if (base == CONV2D_OUT_BF16)
        return out == CONV2D_OUT_BF16 ? start_pass_as<TRANS, VEC, HALVED, B, B>(p, stream) : start_pass_as<TRANS, VEC, HALVED, B, float>(p, stream);
    return out == CONV2D_OUT_BF16 ? start_pass_as<TRANS, VEC, HALVED, float, B>(p, stream) : start_pass_as<TRANS, VEC, HALVED, float, float>(p, stream);
}

template <bool TRANS>
int start_pass(const PassParams& p, int32_t base, int32_t out, bool vec, bool halved, cudaStream_t stream)
{
    if (vec) return halved ? start_pass_by_types<TRANS, true, 1>(p, base, out, stream) : start_pass_by_types<TRANS, true, 0>(p, base, out, stream);
    return halved ? start_pass_by_types<TRANS, false, 1>(p, base, out, stream) : start_pass_by_types<TRANS, false, 0>(p, base, out, stream);
}

}  // namespace ad
}  // namespace sgb
