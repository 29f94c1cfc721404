// One direction through the adapters, in [rows][from] -> mid [rows][rank] -> out [rows][to], by tiles of up to 128 rows of one adapter:
//
//   mid = scale * in w1^T,  out = act(base + mid w2^T)
//
// Forward w1 is a[e] and w2 is b[e], both K-major operands; backward (TRANS) w1 is b[e]^T and w2 a[e]^T, both MN-major.
//
// in, base and out each pass once over HBM and bind it: with rank r the matrix units have 2r flops to some 4 bytes.  What is reached is less, as a CTA's parts
// follow one another: 8192 x 4096 -> 4096 of rank 64 takes 53 to 57 us (33 at HBM's rate, 3.9 to 4.1 TB/s), 12544 x 256 -> 1024 of rank 16, y fp32, 23 to 24 us (12.5).  A cluster
// of S CTAs shares a tile: each takes a part of `from` for the first product, 128/S rows of the join and a part of `to` for the
// second.  One CTA fills an SM: what HBM needs in flight are bytes, and 96 KB of base on their way to shared memory gave more than two CTAs with
// theirs in registers.  mid never leaves the chip but for the copy that the gradients need.
//
// First product: rows of `in` are gathered by the plan's order with cp.async, 128 bytes of a row at a time, 128 x rank x 128 a stage (the loop around a stage costs its warps some
// 600 clocks, more than its copies of half the size).  The sums over
// the parts meet in shared memory as fp32, are joined in the CTAs' order and cut into three bf16 parts that
// hold all 24 bits: the second product, K = 3 * rank, is that of an fp32 mid.
//
// Second product: mid's parts are its A operand in tensor memory (from shared memory they would be read once for each chunk and take
// most of its bandwidth), 128 columns of `to` its B.  Two groups of 8 warps finish chunks by turns, each with an accumulator of its own.  A thread reads the accumulator in the 16 x 256-bit layout, 2
// neighbouring columns of a lane in each group of 8; w2's rows are placed in shared memory in an order that makes these 8 (fp32: 4) neighbouring columns of out, so base and
// out move in 16-byte vectors, base three turns ahead by way of a ring that each thread alone reads.
//
// Rows that are not whole vectors (VEC = false) come through registers without running ahead, and are finished one row at a time: 777 x 1001 -> 2001
// of rank 20 takes 20 us, most of it latency (1.7 at HBM's rate).
//
// Every wait is bounded.  A thread whose wait has run out waits no more and goes on with whatever is in memory: the status word is set, and what the call
// stores, within its results, is undefined.  It waits again, as long at most, for what its cluster sends it, and the CTA for its MMAs, before the memory that these read and
// write is given up.
#pragma once

#include "adapter_params.cuh"
#include "adapter_ptx.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

constexpr int P_W2_WARPS = 3, P_W2_THREADS = 32 * P_W2_WARPS;  // that bring w2's chunks
constexpr int P_THREADS = P_LOADERS + 32 + P_W2_THREADS;
constexpr uint32_t P_TMEM = 512;  // the first product's sums, then 256 columns of chunks; mid's parts at the end

template <bool TRANS, bool VEC, int HALVED, typename TB, typename TO>
struct Pass {
    static constexpr int ROWS = TILE >> HALVED;  // of a tile
    static constexpr int COLS = P_COLS, BUFS = 2;  // of `to`, in a chunk; accumulators of chunks, one to each group
    static constexpr int LANES = 32 >> HALVED;   // of a warp's 32 lanes of tensor memory that hold rows

    const PassParams& p;
    const PassSmem s;
    uint8_t* mem;
    uint64_t *full, *empty, *done, *w2_full, *w2_empty, *d_full, *d_empty, *mid_full, *last;
    int* ids;  // numbers of the tile's rows
    uint32_t* slot;
    int tid, warp, lane, rank_in, e, n_stages, n_bufs;
    int group;  // of two that finish chunks by turns

    Piece piece;

    __device__ __forceinline__ Pass(const PassParams& p, uint8_t* raw) : p(p), s(p.rank), mem(raw)
    {
        n_stages = s.stages();
        n_bufs = s.buffers();
        full = reinterpret_cast<uint64_t*>(raw + s.area() + s.chunk());
        empty = full + P_MOST_STAGES;
        done = empty + P_MOST_STAGES;
        w2_full = done + 1;
        w2_empty = w2_full + P_MOST_CHUNKS;
        d_full = w2_empty + P_MOST_CHUNKS;
        d_empty = d_full + BUFS;
        mid_full = d_empty + BUFS;
        last = mid_full + 1;
        ids = reinterpret_cast<int*>(last + 1);
        slot = reinterpret_cast<uint32_t*>(ids + TILE);
        tid = threadIdx.x;
        warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, as the compiler then knows
        lane = tid & 31;
        rank_in = blockIdx.x % p.splits;
        group = warp >> 3;
    }
    // Once a wait has run out, `ok` is false and the thread waits no more.  (Reported at the thread's end instead, it cost loaders of rows that are not whole
    // vectors up to 7%.)
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& ok) const
    {
        if (!ptx::mbar_try_wait(bar, parity) && ok && !ptx::mbar_wait(bar, parity, WAIT_NS)) {
            ok = false;
            atomicMax(p.status, 6u);
        }
    }
    __device__ __forceinline__ float* mids() const { return reinterpret_cast<float*>(mem + s.area() - s.sums()); }
    __device__ __forceinline__ uint8_t* w2_buf(int i) const { return i ? mem + s.area() - s.ring() - i * s.chunk() : mem + s.area(); }
    __device__ __forceinline__ uint32_t base_ring() const { return ptx::smem_addr(mem) + s.area() - s.ring() + 16 * tid; }

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

    // Where a loader's copies of an MN-major w1 go: 64 rows of rank/8 16-byte columns, one after another in memory.
    // (Addresses are kept in registers: computed for each copy they cost the loaders more time than the copies.)
    static constexpr int PLACES = 64 * MOST_RANK / 8 / P_LOADERS;
    uint32_t place[PLACES];
    __device__ __forceinline__ void make_places()
    {
        const int per = p.rank >> 3;
#pragma unroll
        for (int j = 0; j < PLACES; ++j) {
            const int i = tid + P_LOADERS * j, row = i / per, c8 = i - row * per;
            place[j] = row >= 64 ? 0xffffffffu : (row & 7) * 16 + (row >> 3) * 128 + c8 * W1_COLUMN;
        }
    }

    // Columns f0 .. f0+63 of the tile's rows and of w1.  rows: at this thread's 16-byte column of every 64th row, w: where its copies of
    // w1 begin, both at column f0.
    __device__ __forceinline__ void load_block(uint32_t at, int f0, const __nv_bfloat16* const (&rows)[ROWS / 64], const __nv_bfloat16* w) const
    {
        const uint32_t w_at = at + TILE * P_BLOCK * 2;
        const int row = tid >> 3, c8 = tid & 7;
        const uint32_t swizzled = (c8 ^ (row & 7)) << 4, mine = lane_of(row) * 128 + swizzled;  // 128-byte swizzle
        if (VEC && f0 + P_BLOCK <= p.from) {
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i)
                ptx::cp_async_16_if(at + mine + 8192 * i, rows[i], row + 64 * i < piece.rows);
            if constexpr (!TRANS) {
                ptx::cp_async_16_if(w_at + row * 128 + swizzled, w, row < p.rank);
                ptx::cp_async_16_if(w_at + row * 128 + swizzled + 8192, w + 64 * static_cast<int64_t>(p.from), row + 64 < p.rank);
            } else {
#pragma unroll
                for (int i = 0; i < PLACES; ++i)
                    ptx::cp_async_16_if(w_at + place[i], w + 8 * P_LOADERS * i, place[i] != 0xffffffffu);
            }
            return;
        }
        // Through registers, all of them on their way at once: rows that are not whole vectors, and the last columns.
        constexpr int MOST = ROWS / 64 + MOST_RANK / 64;
        uint32_t v[MOST][4], to[MOST];
        const __nv_bfloat16* first = p.w1 + e * (static_cast<int64_t>(p.rank) * p.from);
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            const __nv_bfloat16* src;
            int left;
            if (i < ROWS / 64) {
                src = rows[i < ROWS / 64 ? i : 0];
                left = row + 64 * i < piece.rows ? p.from - f0 - 8 * c8 : 0;
                to[i] = row + 64 * i < piece.rows ? at + mine + 8192 * i : 0u;
            } else if constexpr (!TRANS) {
                const int r = row + 64 * (i - ROWS / 64);
                src = first + static_cast<int64_t>(r) * p.from + f0 + 8 * c8;
                left = r < p.rank ? p.from - f0 - 8 * c8 : 0;
                to[i] = r < p.rank ? w_at + r * 128 + swizzled : 0u;
            } else {  // 64 rows of rp/8 16-byte columns
                const int j = tid + P_LOADERS * (i - ROWS / 64), k = (j >> 1) & 63, n8 = 2 * (j >> 7) + (j & 1);
                src = first + static_cast<int64_t>(f0 + k) * p.rank + 8 * n8;
                left = j < s.rp * 8 && f0 + k < p.from ? p.rank - 8 * n8 : 0;
                to[i] = j < s.rp * 8 ? w_at + (k & 7) * 16 + n8 * W1_COLUMN + (k >> 3) * 128 : 0u;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = 0u;
            if (left > 0) mx::load_any<4, 2>(v[i], src, left < 8 ? 2 * left : 16);
        }
#pragma unroll
        for (int i = 0; i < MOST; ++i)
            if (to[i]) ptx::st_shared_v4(to[i], v[i][0], v[i][1], v[i][2], v[i][3]);
        if (VEC) ptx::fence_proxy_async_smem();
    }

    // A thread finishes vectors of 8 elements, of 32 columns: one run of 8 or, where base or out has 32 bits, two of 4 at 16 columns' distance, so that
    // four threads' runs are whole sectors (rows that are not whole vectors: finish_rows).
    // It gets columns 8j + 2(lane%4) + {0, 1} of the accumulator, j = 0 .. 3; w2's column c becomes row place_of(c) of the operand for that.
    static constexpr int RUN = sizeof(TB) == 2 && sizeof(TO) == 2 ? 8 : 4, RUNS = 8 / RUN, APART = 4 * RUN;
    __device__ __forceinline__ static int place_of(int c)
    {
        if constexpr (!VEC) return c;
        return (c & ~31) + (c & 1) + (RUN == 8 ? 8 * ((c >> 1) & 3) + 2 * ((c >> 3) & 3) : 8 * (2 * ((c >> 4) & 1) + ((c >> 1) & 1)) + 2 * ((c >> 2) & 3));
    }
    // w2's columns of a chunk from c0 on, by the warps that bring it.
    __device__ __forceinline__ void load_w2(uint8_t* buf, int c0) const
    {
        const int64_t size = static_cast<int64_t>(p.rank) * p.to;
        const __nv_bfloat16* w = p.w2 + e * size;
        const uint32_t at = ptx::smem_addr(buf);
        const int wt = tid - (P_LOADERS + 32), ww = warp - (P_WARPS + 1);
        if (VEC && c0 + COLS <= p.to) {
            if constexpr (!TRANS) {
                // as many threads to a column's ranks as a power of two covers them
                const int per = p.rank >> 3, shift = per <= 1 ? 0 : 32 - __clz(per - 1), step = P_W2_THREADS >> shift;
                const int c8 = wt & ((1 << shift) - 1);
                const uint32_t dst = at + c8 * s.column();
                const __nv_bfloat16* src = w + static_cast<int64_t>(c0 + (wt >> shift)) * p.rank + 8 * c8;
#pragma unroll 4
                for (int c = wt >> shift; c < COLS; c += step, src += step * p.rank) {
                    const int n = place_of(c);
                    ptx::cp_async_16_if(dst + (n & 7) * 16 + (n >> 3) * 144, src, c8 < per);
                }
            } else {
                const int c = 2 * lane, n = place_of(c);
                const uint32_t dst = at + (n & 7) * 2 + (n >> 3) * 144;
                const __nv_bfloat16* src = w + static_cast<int64_t>(ww) * p.to + c0 + c;
#pragma unroll 4
                for (int k = ww; k < p.rank; k += P_W2_WARPS, src += P_W2_WARPS * static_cast<int64_t>(p.to)) {
                    const uint32_t to = dst + (k & 7) * 16 + (k >> 3) * s.column();
                    ptx::cp_async_4_if(to, src, true);
                    ptx::cp_async_4_if(to + 8 * 144, src + 64, true);
                }
            }
        } else {
            // 8 elements of a row of w2 at a time through registers, BATCH of them on their way at once
            constexpr int BATCH = 4;
            const int all = s.rp * COLS / 8, per = TRANS ? COLS / 8 : s.rp >> 3;
            for (int i0 = wt; i0 < all; i0 += BATCH * P_W2_THREADS) {
                uint32_t v[BATCH][4];
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int i = i0 + u * P_W2_THREADS, line = i / per, at8 = 8 * (i - line * per);  // a column's 8 ranks, or a rank's 8 columns
                    const int left = i >= all ? 0 : TRANS ? (line < p.rank ? p.to - c0 - at8 : 0) : c0 + line < p.to ? p.rank - at8 : 0;
                    const __nv_bfloat16* src = TRANS ? w + static_cast<int64_t>(line) * p.to + c0 + at8 : w + static_cast<int64_t>(c0 + line) * p.rank + at8;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[u][k] = 0u;
                    if (left > 0) mx::load_any<4, 2>(v[u], src, left < 8 ? 2 * left : 16);
                }
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int i = i0 + u * P_W2_THREADS, line = i / per, at8 = 8 * (i - line * per);
                    if (i >= all) break;
                    if constexpr (TRANS) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int n = place_of(at8 + 2 * k);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (line & 7) * 16 + (n & 7) * 2 + (n >> 3) * 144 + (line >> 3) * s.column()), "r"(v[u][k]) : "memory");
                        }
                    } else {
                        const int n = place_of(line);
                        ptx::st_shared_v4(at + (n & 7) * 16 + (n >> 3) * 144 + (at8 >> 3) * s.column(), v[u][0], v[u][1], v[u][2], v[u][3]);
                    }
                }
            }
            if (VEC) ptx::fence_proxy_async_smem();
        }
    }
    // The part of a chunk of w2 that pads an odd number of 8 ranks; whole copies do not reach it.
    __device__ __forceinline__ void clear_pad(uint8_t* buf) const
    {
        if constexpr (!VEC) return;
        if (!(p.rank & 8)) return;
        for (int i = tid - (P_LOADERS + 32); i < COLS; i += P_W2_THREADS)
            ptx::st_shared_v4(ptx::smem_addr(buf) + (i & 7) * 16 + (i >> 3) * 144 + (p.rank >> 3) * s.column(), 0u, 0u, 0u, 0u);
        ptx::fence_proxy_async_smem();
    }
    // w2's chunk j (columns from c0 on), when its buffer is free.
    __device__ __forceinline__ void bring_w2(int j, int c0, bool& ok) const
    {
        const int buf = j % n_bufs;
        wait(&w2_empty[buf], (static_cast<uint32_t>(j / n_bufs) & 1u) ^ 1u, ok);
        if (j < n_bufs) clear_pad(w2_buf(buf));
        load_w2(w2_buf(buf), c0);
        ptx::cp_async_commit();
    }

    // This CTA's rows of the sums over the cluster: scaled, to mid, and on to every CTA.
    template <int S>
    __device__ __forceinline__ void join(const float* sums, float scale) const
    {
        constexpr int SHARE = ROWS / S;
        const int eighths = s.rp >> 3;
        for (int i = tid < P_LOADERS ? tid : SHARE * eighths; i < SHARE * eighths; i += P_LOADERS) {  // neighbouring lanes read neighbouring parts of a row
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

    // A thread finishes eight vectors (four of a halved tile) of a chunk, two side by side at 32 columns' distance in each of its rows, 8 rows apart.  It holds HOLD of them at a time, a turn: 64 bytes of base.
    static constexpr int MINE = 4 >> HALVED, VECTORS = 2 * MINE;  // rows of a thread
    static constexpr int HOLD = sizeof(TB) == 2 ? 4 : 2, TURNS = VECTORS / HOLD, WORDS = 2 * sizeof(TB);
    struct Held {
        uint32_t u[HOLD][WORDS];
    };
    const TB* base_at[MINE];
    TO* out_at[MINE];
    __device__ __forceinline__ static constexpr int row_index(int i) { return i % MINE; }
    __device__ __forceinline__ static constexpr int side_of(int i) { return i / MINE; }
    __device__ __forceinline__ int row_of(int i) const { return LANES * (warp & 3) + (lane >> 2) + 8 * row_index(i); }
    __device__ __forceinline__ int col_of(int i, int c0) const { return c0 + 64 * ((warp >> 2) & 1) + 32 * side_of(i) + RUN * (lane & 3); }
    __device__ __forceinline__ void make_rows()
    {
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int64_t t = ids[row_of(i)];
            row_here[i] = row_of(i) < piece.rows;
            base_here[i] = row_here[i] && p.base;
            base_at[i] = static_cast<const TB*>(p.base) + t * p.base_stride + col_of(i, 0);
            out_at[i] = static_cast<TO*>(p.out) + t * p.out_stride + col_of(i, 0);
        }
    }
    bool row_here[MINE], base_here[MINE];  // the thread's rows are of the tile; and there is a base
    // Turn `turn` of the chunk at c0, on its way to slot `slot` of the thread's ring (which no other thread reads: it has no barrier); `whole`: all
    // the chunk's columns exist.
    static constexpr int PIECE = RUN * sizeof(TB);  // bytes of a run of base
    __device__ __forceinline__ void ask_base(int slot, int turn, int c0, bool whole, bool wanted) const
    {
        if constexpr (VEC) {
            const uint32_t at = base_ring() + slot * (P_LOADERS * 64) - tid * (16 - PIECE);
#pragma unroll
            for (int k = 0; k < HOLD; ++k) {
                const int side = (turn * HOLD + k) / MINE;
                const bool upper = HOLD < MINE && (turn & 1);  // rows 2 and 3 of four
                const TB* src = (upper ? base_at[(k + HOLD) % MINE] : base_at[k % MINE]) + c0 + 32 * side;
                const bool here = wanted && (upper ? base_here[(k + HOLD) % MINE] : base_here[k % MINE]);
#pragma unroll
                for (int r = 0; r < RUNS; ++r) {
                    const bool in = here && (whole || col_of(0, c0) + 32 * side + APART * r < p.to);
                    const uint32_t dst = at + (k * RUNS + r) * (P_LOADERS * PIECE);
                    if constexpr (PIECE == 16)
                        ptx::cp_async_16_if(dst, src + APART * r, in);
                    else
                        ptx::cp_async_8_if(dst, src + APART * r, in);
                }
            }
        }
    }
    __device__ __forceinline__ void get_base(Held& b, int slot) const
    {
        if constexpr (VEC) {
            const uint32_t at = base_ring() + slot * (P_LOADERS * 64) - tid * (16 - PIECE);
#pragma unroll
            for (int i = 0; i < HOLD * RUNS; ++i) {
                constexpr int W = PIECE / 4;
                uint32_t* to = b.u[i / RUNS] + i % RUNS * W;
                if constexpr (PIECE == 16) {
                    const uint4 q = ptx::ld_shared_v4(at + i * (P_LOADERS * 16));
                    to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                } else {
                    const uint2 q = ptx::ld_shared_v2(at + i * (P_LOADERS * 8));
                    to[0] = q.x, to[1] = q.y;
                }
            }
        }
    }
    // The same straight from memory.
    __device__ __forceinline__ void load_base(Held& b, int turn, int c0) const
    {
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i = turn * HOLD + k;
            TB* v = reinterpret_cast<TB*>(b.u[k]);
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                const TB* src = base_at[row_index(i)] + c0 + 32 * side_of(i) + APART * r;
                const int left = base_here[row_index(i)] ? p.to - col_of(i, c0) - APART * r : 0;
#pragma unroll
                for (int j = 0; j < RUN; ++j) v[r * RUN + j] = j < left ? src[j] : TB(0.f);
            }
        }
    }
    // out = act(base + sum) for a turn: `v` the sums of the four vectors that it belongs to, as they come from tensor memory.
    __device__ __forceinline__ void finish(const Held& b, const uint32_t (&v)[2][16], int turn, int c0, bool whole, bool live) const
    {
        float2 f[HOLD][4];
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i = turn * HOLD + k;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 sum = make_float2(__uint_as_float(v[i >> 1 & 1][4 * j + 2 * (i & 1)]), __uint_as_float(v[i >> 1 & 1][4 * j + 2 * (i & 1) + 1]));
                const float2 base = !p.base ? make_float2(0.f, 0.f) : sizeof(TB) == 2 ? make_float2(__uint_as_float(b.u[k][j] << 16), __uint_as_float(b.u[k][j] & 0xffff0000u))
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
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                TO* row = out_at[row_index(i)] + c0 + 32 * side_of(i) + APART * r;
                const float2* from = f[k] + r * (RUN / 2);
                const int col = col_of(i, c0) + APART * r;
                const bool here = live && row_here[row_index(i)];
                if constexpr (sizeof(TO) == 4) {
                    ptx::st_stream_v4_if(row, make_uint4(__float_as_uint(from[0].x), __float_as_uint(from[0].y), __float_as_uint(from[1].x), __float_as_uint(from[1].y)),
                                         here && (whole || col < p.to));
                } else {
                    uint32_t o[RUN / 2];
#pragma unroll
                    for (int j = 0; j < RUN / 2; ++j) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(from[j].x, from[j].y);
                        o[j] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    if constexpr (RUN == 8)
                        ptx::st_stream_v4_if(row, make_uint4(o[0], o[1], o[2], o[3]), here && (whole || col < p.to));
                    else
                        ptx::st_stream_v2_if(row, make_uint2(o[0], o[1]), here && (whole || col < p.to));
                }
            }
        }
    }

    // Rows that are not whole vectors: the warp's rows of 64 columns of the chunk at c0 one after another, 32 neighbouring elements at a time, one to a lane (in
    // the accumulator's own order 8 rows' elements took 8 turns of a load or store: 12867 x 296 -> 659 56 us), by way of the warp's share of the ring.
    // `at`: the warp's 64 columns of tensor memory, if there are sums.
    static constexpr int BATCH = 16;
    __device__ __forceinline__ void ask_rows(float (&b)[BATCH], int first, int col) const
    {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int row = LANES * (warp & 3) + first + i;
            b[i] = 0.f;
            if (p.base && row < piece.rows && col < p.to) b[i] = mx::to_float(static_cast<const TB*>(p.base)[ids[row] * p.base_stride + col]);
        }
    }
    template <bool SUMS, typename Wait, typename Free>
    __device__ __forceinline__ void finish_rows(uint32_t at, int c0, bool live, const Wait& wait_sums, const Free& free_sums) const
    {
        constexpr int PARTS = 2 * LANES / BATCH;  // batches of rows of both halves of the columns
        float b[2][BATCH];
        const int col0 = c0 + 64 * ((warp >> 2) & 1) + lane;
        ask_rows(b[0], 0, col0);
        wait_sums();
        float* mine = reinterpret_cast<float*>(mem + s.area() - s.ring() + warp * (s.ring() / P_WARPS));  // [LANES][33]
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const int half = k / (PARTS / 2), first = k % (PARTS / 2) * BATCH, col = col0 + 32 * half;
            if (k + 1 < PARTS) ask_rows(b[(k + 1) & 1], (k + 1) % (PARTS / 2) * BATCH, col0 + 32 * ((k + 1) / (PARTS / 2)));
            if (SUMS && first == 0) {
                uint32_t v[2][16];
                ptx::tmem_ld_32x32b_x16(at + 32 * half, v[0]);
                ptx::tmem_ld_32x32b_x16(at + 32 * half + 16, v[1]);
                ptx::tmem_ld_wait();
                if (half) free_sums();
                __syncwarp();
                if (lane < LANES)
#pragma unroll
                    for (int c = 0; c < 32; ++c) mine[lane * 33 + c] = __uint_as_float(v[c >> 4][c & 15]);
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = LANES * (warp & 3) + first + i;
                float f = b[k & 1][i] + (SUMS ? mine[(first + i) * 33 + lane] : 0.f);
                if (p.relu) f = __uint_as_float(ptx::relu_nan(__float_as_uint(f)));
                if (live && row < piece.rows && col < p.to) mx::from_float(static_cast<TO*>(p.out)[ids[row] * p.out_stride + col], f);
            }
        }
    }

    // Base's first chunks to L2, where HBM works on them while the sums are joined.
    static constexpr int AHEAD = sizeof(TB) == 4 ? 4 : 2;
    __device__ __forceinline__ void prefetch_base(int chunk0, int chunk1) const
    {
        constexpr int LINES = AHEAD * COLS * sizeof(TB) / 128, EACH = 128 / sizeof(TB);
        if (!p.base || !p.out) return;
        for (int i = tid; i < piece.rows * LINES; i += P_LOADERS) {
            const int row = i / LINES, c = chunk0 * COLS + (i - row * LINES) * EACH;
            if (c < p.to && c < chunk1 * COLS) ptx::prefetch_l2(static_cast<const TB*>(p.base) + ids[row] * p.base_stride + c);
        }
    }

    // Rows without an adapter: out = act(base), mid = 0.
    __device__ __forceinline__ void without(int chunk0, int chunk1) const
    {
        if (p.mid && rank_in == 0)
            for (int i = tid; i < piece.rows * p.rank; i += P_THREADS)
                p.mid[static_cast<int64_t>(ids[i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (!p.out || warp >= P_WARPS) return;
        for (int c = chunk0 + group; c < chunk1; c += 2) {
            if constexpr (!VEC) {
                finish_rows<false>(0u, c * COLS, true, [] {}, [] {});
            } else {
#pragma unroll
                for (int turn = 0; turn < TURNS; ++turn) {
                    Held b;
                    load_base(b, turn, c * COLS);
                    const uint32_t none[2][16] = {};
                    finish(b, none, turn, c * COLS, false, true);
                }
            }
        }
    }

    __device__ __forceinline__ void run()
    {
        if (tid == 0) {
            for (int i = 0; i < n_stages; ++i) {
                ptx::mbar_init(&full[i], i == 0 ? P_WARPS + LOST_ROWS : P_WARPS);
                ptx::mbar_init(&empty[i], 1);
            }
            ptx::mbar_init(done, 1 + LOST_DONE);
            for (int i = 0; i < n_bufs; ++i) {
                ptx::mbar_init(&w2_full[i], P_W2_WARPS);
                ptx::mbar_init(&w2_empty[i], 1);
            }
            for (int i = 0; i < BUFS; ++i) {
                ptx::mbar_init(&d_full[i], 1);
                ptx::mbar_init(&d_empty[i], P_WARPS / 2);
            }
            ptx::mbar_init(mid_full, 1);
            ptx::mbar_init(last, 1);
            if (p.splits > 1) ptx::mbar_arrive_expect_tx(mid_full, (ROWS - ROWS / p.splits) * s.pitch() * 4);
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
        if (p.early) ptx::grid_launch_dependents();
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
            if (VEC && warp < P_WARPS) make_rows();
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
        const int n = chunk1 - chunk0;
        bool ok = true;
        const float scale = p.scale ? __ldg(p.scale + e) : 1.f;
        if (warp < P_WARPS) {
            const __nv_bfloat16* rows[ROWS / 64];
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i) rows[i] = p.in + ids[(tid >> 3) + 64 * i] * p.in_stride + 8 * (tid & 7) + s0 * P_STEP;
            const __nv_bfloat16* w = p.w1 + e * (static_cast<int64_t>(p.rank) * p.from) +
                                     (TRANS ? static_cast<int64_t>(s0 * P_STEP) * p.rank + 8 * tid : static_cast<int64_t>(tid >> 3) * p.from + 8 * (tid & 7) + s0 * P_STEP);
            const int64_t w_step = TRANS ? P_BLOCK * p.rank : P_BLOCK;
            if (VEC) make_places();
            constexpr int LAG = VEC ? 1 : 0;  // stages on their way behind the one that is asked for
            int at = 0, told = 0;
            uint32_t free_phase = 1u;
            for (int it = 0; it < s1 - s0; ++it) {
                wait(&empty[at], free_phase, ok);
                const uint32_t st = ptx::smem_addr(mem) + at * s.stage();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int f0 = (s0 + it) * P_STEP + h * P_BLOCK;
                    if (f0 < p.from) load_block(st + h * s.block(), f0, rows, w);
#pragma unroll
                    for (int i = 0; i < ROWS / 64; ++i) rows[i] += P_BLOCK;
                    w += w_step;
                }
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
        } else if (warp == P_WARPS) {
            int at = 0, acc = 0;
            uint32_t phase = 0u, again = 0u;
            for (int it = 0; it < s1 - s0; ++it) {
                wait(&full[at], phase, ok);
                __syncwarp();  // what follows is the whole warp's
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((s0 + it) * P_STEP + h * P_BLOCK >= p.from) break;
                    const uint32_t a = ptx::smem_addr(mem) + at * s.stage() + h * s.block(), b = a + TILE * P_BLOCK * 2;
                    ptx::mma_bf16_elect_x4(tmem + acc * s.rp, ptx::sw128_kmajor_desc(a), TRANS ? ptx::plain_mnmajor_desc(b, 128, W1_COLUMN) : ptx::sw128_kmajor_desc(b),
                                           32 / 16, (TRANS ? 256 : 32) / 16, TRANS ? ptx::idesc_bf16_f32_bmn(TILE, s.rp) : ptx::idesc_bf16_f32(TILE, s.rp), again);
                    acc = acc + 1 == s.accumulators() ? 0 : acc + 1;
                    again = acc ? again : 1u;
                }
                ptx::mma_commit_elect(&empty[at]);
                at = at + 1 == n_stages ? 0 : at + 1;
                phase = at ? phase : phase ^ 1u;
            }
            ptx::mma_commit_elect(done);
        } else if (n > 0) {
            bring_w2(0, chunk0 * COLS, ok);
        }
        __syncwarp();
        wait(done, 0, ok);
        __syncwarp();
        if (warp > P_WARPS && n > 0) {
            ptx::cp_async_wait_all();
            arrive(&w2_full[0]);
            if (n > 1 && !s.late()) bring_w2(1, (chunk0 + 1) * COLS, ok);
        }
        // The ring is free: the sums.
        float* sums = reinterpret_cast<float*>(mem);
        if (warp < P_WARPS) {
            ptx::tc_fence_after();
            const int row = LANES * (warp & 3) + lane;
            const int blocks = ((s1 * P_STEP < p.from ? s1 * P_STEP : p.from) - s0 * P_STEP + P_BLOCK - 1) / P_BLOCK;
            const int accs = blocks < s.accumulators() ? blocks : s.accumulators();
            for (int c = 16 * (warp >> 2); c < s.rp; c += 64) {
                const uint32_t from = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c;
                float f[16] = {};
                for (int i = 0; i < accs; i += 2) {
                    uint32_t v[2][16];
                    ptx::tmem_ld_32x32b_x16(from + i * s.rp, v[0]);
                    ptx::tmem_ld_32x32b_x16(from + (i + 1 < accs ? i + 1 : i) * s.rp, v[1]);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) f[k] += __uint_as_float(v[0][k]);
                    if (i + 1 < accs)
#pragma unroll
                        for (int k = 0; k < 16; ++k) f[k] += __uint_as_float(v[1][k]);
                }
                const uint32_t at = ptx::smem_addr(sums + row * s.pitch() + c);
                if (lane < LANES)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        ptx::st_shared_v4(at + 4 * i, __float_as_uint(f[i]), __float_as_uint(f[i + 1]), __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3]));
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
        // All of mid is here: none of this CTA's peers reads its sums any more, and what they sent has come.  Every thread waits for that, also after a wait
        // that has run out, as the peers send in any case, and no memory that they send to or from may be given up.
        if (p.splits > 1) {
            if (!ptx::mbar_wait(mid_full, 0, LAST_WAIT_NS)) {
                ok = false;
                atomicMax(p.status, 6u);
            }
            __syncwarp();
            ptx::cluster_arrive_relaxed();
        }
        const uint32_t parts = tmem + P_TMEM - 3 * s.rp / 2;
        if (warp < P_WARPS) {
            store_parts(parts);
            ptx::tc_fence_before();
            if (p.splits > 1) ptx::cluster_wait();  // what this CTA sent has been received: its place is the ring's now
        }
        if (s.late())
            __syncthreads();
        else if (warp <= P_WARPS)
            ptx::named_bar_sync(1, P_LOADERS + 32);  // the warps that bring w2 are not waited for
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
                const uint64_t wd = ptx::plain_kmajor_desc(w, s.column(), 144), w_step = 2 * s.column() / 16;
                const uint32_t idesc = TRANS ? ptx::idesc_bf16_f32_bmn(TILE, COLS) : ptx::idesc_bf16_f32(TILE, COLS);
                const int whole = s.rp / 32;  // of the reduction, in twice three MMAs
                for (int k = 0; k < whole; ++k) ptx::mma_bf16_parts_x2(tmem + COLS * b, parts + 16 * k, wd + 2 * k * w_step, s.rp / 2, w_step, idesc, k > 0);
                if (s.rp & 16) ptx::mma_bf16_parts(tmem + COLS * b, parts + 16 * whole, wd + 2 * whole * w_step, s.rp / 2, idesc, whole > 0);
                ptx::mma_commit_elect(&d_full[b]);
                ptx::mma_commit_elect(&w2_empty[buf]);
                buf = buf + 1 == n_bufs ? 0 : buf + 1;
                phase = buf ? phase : phase ^ 1u;
            }
            // The CTA lives until its MMAs have ended, whatever waits have run out.
            ptx::mma_commit_elect(last);
            if (!ptx::mbar_wait(last, 0, LAST_WAIT_NS)) atomicMax(p.status, 6u);
        } else if (warp > P_WARPS) {
            // the word of each a chunk later
            if (n > 1 && s.late()) bring_w2(1, (chunk0 + 1) * COLS, ok);
            for (int j = 2; j < n; ++j) {
                bring_w2(j, (chunk0 + j) * COLS, ok);
                ptx::cp_async_wait<1>();
                arrive(&w2_full[(j - 1) % n_bufs]);
            }
            ptx::cp_async_wait_all();
            if (n > 1) arrive(&w2_full[(n - 1) % n_bufs]);
        } else if (!VEC) {
            for (int j = group; j < n; j += 2)
                finish_rows<true>(
                    tmem + COLS * group + 64 * ((warp >> 2) & 1) + (static_cast<uint32_t>(32 * (warp & 3)) << 16), (chunk0 + j) * COLS, ok,
                    [&] {
                        wait(&d_full[group], static_cast<uint32_t>(j >> 1) & 1u, ok);
                        __syncwarp();
                        ptx::tc_fence_after();
                    },
                    [&] {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive_if(&d_empty[group], lane == 0);
                    });
        } else if (group < n) {
            // This group's chunks, every other one; base P_DEPTH turns ahead.
            const auto ask = [&](int slot, int j, int t) {  // turn t from chunk j's beginning on
                const int c = j + 2 * (t / TURNS), c0 = (chunk0 + c) * COLS;
                ask_base(slot, t % TURNS, c0, c0 + COLS <= p.to, c < n);
                ptx::cp_async_commit();
            };
#pragma unroll
            for (int t = 0; t < P_DEPTH; ++t) ask(t, group, t);
            int slot = 0;
            for (int j = group; j < n; j += 2) {
                const int c0 = (chunk0 + j) * COLS;
                const bool whole = c0 + COLS <= p.to;
                wait(&d_full[group], static_cast<uint32_t>(j >> 1) & 1u, ok);
                __syncwarp();
                ptx::tc_fence_after();
                const uint32_t at = tmem + COLS * group + 64 * ((warp >> 2) & 1) + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
#pragma unroll
                for (int q = 0; q < VECTORS / 4; ++q) {
                    uint32_t v[2][16];
                    ptx::tmem_ld_16x256b_x4(at + 32 * q, v[0]);
                    ptx::tmem_ld_16x256b_x4(at + (HALVED ? 32u : 32 * q + (16u << 16)), v[1]);
                    ptx::tmem_ld_wait();
                    if (q + 1 == VECTORS / 4) {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive_if(&d_empty[group], lane == 0);
                    }
#pragma unroll
                    for (int h = 0; h < 4 / HOLD; ++h) {
                        const int t = q * (4 / HOLD) + h;
                        ptx::cp_async_wait<P_DEPTH - 1>();
                        Held held;
                        get_base(held, slot);
                        finish(held, v, t, c0, whole, ok);
                        ask(slot, j, t + P_DEPTH);  // what the slot held is in registers
                        slot = slot + 1 == P_DEPTH ? 0 : slot + 1;
                    }
                }
            }
        }
        __syncwarp();
        ptx::cp_async_wait_all();
        __syncwarp();
        if (p.splits > 1 && warp >= P_WARPS) ptx::cluster_wait();
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
