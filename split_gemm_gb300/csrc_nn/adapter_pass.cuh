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
// Second product: 64 columns of `to` at a time, two accumulators in turn.  A thread reads the accumulator in the 16 x 256-bit layout, 2
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

constexpr int P_WARPS = 8, P_LOADERS = 32 * P_WARPS, P_THREADS = P_LOADERS + 32;
constexpr uint64_t P_WAIT_NS = 1000000000ull;
constexpr uint32_t P_TMEM = 256;  // rank and two chunks

template <bool TRANS, bool VEC, typename TB, typename TO>
struct Pass {
    const PassParams& p;
    const PassSmem s;
    uint8_t* mem;
    uint64_t *full, *empty, *done, *w2_full, *d_full, *d_empty;
    uint32_t* slot;
    volatile uint32_t* abort_flag;
    int tid, warp, lane, rank_in, e;
    Piece piece;

    __device__ __forceinline__ Pass(const PassParams& p, uint8_t* raw) : p(p), s(p.rank, p.stages), mem(raw)
    {
        full = reinterpret_cast<uint64_t*>(raw + s.ring() + s.parts() + s.chunk());
        empty = full + P_MOST_STAGES;
        done = empty + P_MOST_STAGES;
        w2_full = done + 1;
        d_full = w2_full + 2;
        d_empty = d_full + 2;
        slot = reinterpret_cast<uint32_t*>(d_empty + 2);
        abort_flag = slot + 1;
        tid = threadIdx.x;
        warp = tid >> 5;
        lane = tid & 31;
        rank_in = blockIdx.x % p.splits;
    }
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, bool& ok) const
    {
        if (ok && !ptx::mbar_wait(bar, parity, P_WAIT_NS)) {
            ok = false;
            *abort_flag = 1u;
        }
        return ok;
    }
    __device__ __forceinline__ uint8_t* parts() const { return mem + s.ring(); }
    __device__ __forceinline__ uint8_t* w2_buf(int i) const { return i ? mem + s.sums() : mem + s.ring() + s.parts(); }

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
    // This thread's part of what `bar` counts is there.
    __device__ __forceinline__ void arrive(uint64_t* bar) const
    {
        if constexpr (VEC) {
            ptx::cp_async_arrive_noinc(bar);
        } else {
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(bar);
        }
    }

    // Where a loader's copies of an MN-major w1 or a K-major w2 go: 64 rows of rank/8 16-byte columns, one after another in memory.
    // (Addresses are kept in registers: computed for each copy they cost the loaders more time than the copies.)
    uint32_t place[4];
    __device__ __forceinline__ void make_places()
    {
        const int per = p.rank >> 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = tid + P_LOADERS * j, row = i / per, c8 = i - row * per;
            const int n = (row & 32) + 8 * ((row >> 1) & 3) + 2 * ((row >> 3) & 3) + (row & 1);  // of w2, as below
            place[j] = row >= 64 ? 0xffffffffu : TRANS ? (row & 7) * 16 + (row >> 3) * 128 + c8 * W1_COLUMN : (n & 7) * 16 + (n >> 3) * 144 + c8 * 1152;
        }
    }

    // Columns f0 .. f0+63 of the tile's rows and of w1.  rows: at this thread's 16-byte column of every 32nd row.
    __device__ __forceinline__ void load_stage(uint8_t* st, int f0, const __nv_bfloat16* const (&rows)[4]) const
    {
        const uint32_t at = ptx::smem_addr(st), w_at = at + TILE * P_STEP * 2;
        const int64_t size = static_cast<int64_t>(p.rank) * p.from;
        const __nv_bfloat16* w = p.w1 + e * size;
        const int row = tid >> 3, c8 = tid & 7;
        const uint32_t mine = row * 128 + ((c8 ^ (row & 7)) << 4);  // 128-byte swizzle
        if (VEC && f0 + P_STEP <= p.from) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (row + 32 * i < piece.rows) ptx::cp_async_16s(at + mine + 4096 * i, rows[i] + f0, 16);
            if constexpr (!TRANS) {
                const __nv_bfloat16* src = w + static_cast<int64_t>(row) * p.from + f0 + 8 * c8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (row + 32 * i < p.rank) ptx::cp_async_16s(w_at + mine + 4096 * i, src, 16);
                    src += 32 * static_cast<int64_t>(p.from);
                }
            } else {
                const __nv_bfloat16* src = w + static_cast<int64_t>(f0) * p.rank + 8 * tid;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (place[i] != 0xffffffffu) ptx::cp_async_16s(w_at + place[i], src + 8 * P_LOADERS * i, 16);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + 32 * i < piece.rows) copy8(at + mine + 4096 * i, rows[i] + f0, p.from - f0 - 8 * c8);
        if constexpr (!TRANS) {
            for (int r = row; r < p.rank; r += 32)
                copy8(w_at + r * 128 + ((c8 ^ (r & 7)) << 4), w + static_cast<int64_t>(r) * p.from + f0 + 8 * c8, p.from - f0 - 8 * c8);
        } else {
            for (int i = tid; i < s.rp * 8; i += P_LOADERS) {  // 64 rows of rp/8 16-byte columns
                const int k = (i >> 1) & 63, n8 = 2 * (i >> 7) + (i & 1);
                const int left = f0 + k < p.from ? p.rank - 8 * n8 : 0;
                copy8(w_at + (k & 7) * 16 + n8 * W1_COLUMN + (k >> 3) * 128, w + static_cast<int64_t>(f0 + k) * p.rank + 8 * n8, left);
            }
        }
    }

    // w2's 64 columns from c0 on: column c of 32 becomes row 8((c>>1)&3) + 2(c>>3) + (c&1) of the operand.
    __device__ __forceinline__ void load_w2(uint8_t* buf, int c0) const
    {
        const uint32_t at = ptx::smem_addr(buf);
        const int64_t size = static_cast<int64_t>(p.rank) * p.to;
        const __nv_bfloat16* w = p.w2 + e * size;
        if (VEC && c0 + P_COLS <= p.to) {
            if constexpr (!TRANS) {
                const __nv_bfloat16* src = w + static_cast<int64_t>(c0) * p.rank + 8 * tid;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (place[i] != 0xffffffffu) ptx::cp_async_16s(at + place[i], src + 8 * P_LOADERS * i, 16);
            } else {
                const int c = 2 * lane;
                uint32_t dst = at + warp * 16 + ((c >> 3) & 3) * 4 + (((c >> 1) & 3) + 4 * (c >> 5)) * 144;
                const __nv_bfloat16* src = w + static_cast<int64_t>(warp) * p.to + c0 + c;
                for (int k = warp; k < p.rank; k += 8, dst += 1152, src += 8 * static_cast<int64_t>(p.to)) ptx::cp_async_4(dst, src, 4);
            }
            return;
        }
        if constexpr (!TRANS) {
            for (int i = tid; i < s.rp * 8; i += P_LOADERS) {
                const int n = (i >> 1) & 63, k8 = 2 * (i >> 7) + (i & 1);
                const int c = c0 + (n & 32) + 8 * ((n >> 1) & 3) + 2 * ((n >> 3) & 3) + (n & 1);
                copy8(at + (n & 7) * 16 + (n >> 3) * 144 + k8 * 1152, w + static_cast<int64_t>(c) * p.rank + 8 * k8, c < p.to ? p.rank - 8 * k8 : 0);
            }
        } else {
            for (int i = tid; i < s.rp * 32; i += P_LOADERS) {
                const int k = i >> 5, c = 2 * (i & 31);
                const uint32_t dst = at + (k & 7) * 16 + ((c >> 3) & 3) * 4 + (((c >> 1) & 3) + 4 * (c >> 5)) * 144 + (k >> 3) * 1152;
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
    // The part of a chunk of w2 that pads an odd number of 8 ranks; whole copies do not reach it.
    __device__ __forceinline__ void clear_pad(uint8_t* buf) const
    {
        if (VEC && (p.rank & 8) && tid < 64) ptx::st_shared_v4(ptx::smem_addr(buf) + (tid & 7) * 16 + (tid >> 3) * 144 + (p.rank >> 3) * 1152, 0u, 0u, 0u, 0u);
        if (VEC) ptx::fence_proxy_async_smem();
    }

    // This CTA's rows of the sums over the cluster: scaled, to mid, and in three parts to every CTA.
    template <int S>
    __device__ __forceinline__ void join(const float* sums, float scale) const
    {
        constexpr int SHARE = TILE / S;
        const int eighths = s.rp >> 3;
        for (int i = tid; i < SHARE * eighths; i += P_THREADS) {
            const int row = rank_in * SHARE + i % SHARE, r = 8 * (i / SHARE);
            const float* at = sums + row * s.pitch() + r;
            float v[8] = {};
            if (row < piece.rows) {
#pragma unroll
                for (int h = 0; h < 8; h += 4) {
                    float4 u[S];
#pragma unroll
                    for (int k = 0; k < S; ++k) {
                        if constexpr (S == 1)
                            u[k] = *reinterpret_cast<const float4*>(at + h);
                        else
                            u[k] = ptx::ld_cluster_v4(ptx::mapa_shared(ptx::smem_addr(at + h), k));
                    }
#pragma unroll
                    for (int k = 0; k < S; ++k) {
                        v[h] += u[k].x;
                        v[h + 1] += u[k].y;
                        v[h + 2] += u[k].z;
                        v[h + 3] += u[k].w;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r + j < p.rank ? v[j] * scale : 0.f;
                if (p.mid) {
                    float* mid = p.mid + static_cast<int64_t>(p.plan.order[piece.first + row]) * p.rank + r;
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
            uint32_t part[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[3], b[3];
                split3(v[2 * j], a[0], a[1], a[2]);
                split3(v[2 * j + 1], b[0], b[1], b[2]);
#pragma unroll
                for (int q = 0; q < 3; ++q) part[q][j] = a[q] | b[q] << 16;
            }
            const uint32_t to = ptx::smem_addr(parts()) + (row & 7) * 16 + (row >> 3) * 128;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const uint32_t dst = to + ((q * s.rp + r) >> 3) * 2048;
                if constexpr (S == 1) {
                    ptx::st_shared_v4(dst, part[q][0], part[q][1], part[q][2], part[q][3]);
                } else {
#pragma unroll
                    for (int k = 0; k < S; ++k) ptx::st_cluster_v4(ptx::mapa_shared(dst, k), part[q][0], part[q][1], part[q][2], part[q][3]);
                }
            }
        }
        ptx::fence_proxy_async_all();
    }

    // A thread's rows of a tile are every 8th of its warp's 32, their elements of a chunk of 64 columns 8 of the warp's 32.  It holds
    // ROWS of those rows at a time: 64 bytes of base.
    static constexpr int ROWS = sizeof(TB) == 2 ? 4 : 2, TURNS = 4 / ROWS, WORDS = 2 * sizeof(TB);
    struct Held {
        uint32_t u[ROWS][WORDS];
    };
    const TB* base_at[4];
    TO* out_at[4];
    __device__ __forceinline__ int row_of(int i) const { return 32 * (warp & 3) + (lane >> 2) + 8 * i; }
    __device__ __forceinline__ int col_of(int c0) const { return c0 + 32 * (warp >> 2) + 8 * (lane & 3); }
    __device__ __forceinline__ void make_rows()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = p.plan.order[piece.first + (row_of(i) < piece.rows ? row_of(i) : 0)];
            base_at[i] = static_cast<const TB*>(p.base) + t * p.base_stride + col_of(0);
            out_at[i] = static_cast<TO*>(p.out) + t * p.out_stride + col_of(0);
        }
    }
    // Turn `turn` of the chunk at c0.
    __device__ __forceinline__ void load_base(Held& b, int turn, int c0) const
    {
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int i = turn * ROWS + k;
            const TB* src = base_at[i] + c0;
            const int left = p.base && row_of(i) < piece.rows ? p.to - col_of(c0) : 0;
            if constexpr (VEC) {
#pragma unroll
                for (int j = 0; j < WORDS; j += 4) {
                    uint4 q = make_uint4(0, 0, 0, 0);
                    if (left > 0) q = __ldcs(reinterpret_cast<const uint4*>(src) + j / 4);
                    b.u[k][j] = q.x, b.u[k][j + 1] = q.y, b.u[k][j + 2] = q.z, b.u[k][j + 3] = q.w;
                }
            } else {
                TB* v = reinterpret_cast<TB*>(b.u[k]);
#pragma unroll
                for (int j = 0; j < WORDS; ++j) b.u[k][j] = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) v[j] = src[j];
            }
        }
    }
    // out = act(base + sum) for row i: `base` its base, `v` its sums as they come from tensor memory.
    __device__ __forceinline__ void finish(const uint32_t (&base)[WORDS], float2 (&v)[4], int i, int c0, bool live) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 b = sizeof(TB) == 2 ? make_float2(__uint_as_float(base[j] << 16), __uint_as_float(base[j] & 0xffff0000u))
                                             : make_float2(__uint_as_float(base[2 * j % WORDS]), __uint_as_float(base[(2 * j + 1) % WORDS]));
            v[j] = mx::add2(v[j], b);
        }
        if (p.relu)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(v[j].x < 0.f ? 0.f : v[j].x, v[j].y < 0.f ? 0.f : v[j].y);
        TO* row = out_at[i] + c0;
        const int left = live && row_of(i) < piece.rows ? p.to - col_of(c0) : 0;
        if constexpr (VEC) {
            if (left <= 0) return;
            if constexpr (sizeof(TO) == 4) {
                __stcs(reinterpret_cast<float4*>(row), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
                __stcs(reinterpret_cast<float4*>(row) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
            } else {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x, v[j].y);
                    o[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
                __stcs(reinterpret_cast<uint4*>(row), make_uint4(o[0], o[1], o[2], o[3]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) mx::from_float(row[j], j % 2 ? v[j / 2].y : v[j / 2].x);
        }
    }

    // Rows without an adapter: out = act(base), mid = 0.
    __device__ __forceinline__ void without(int chunk0, int chunk1) const
    {
        if (p.mid && rank_in == 0)
            for (int i = tid; i < piece.rows * p.rank; i += P_THREADS)
                p.mid[static_cast<int64_t>(p.plan.order[piece.first + i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (!p.out || warp >= P_WARPS) return;
        for (int c = chunk0; c < chunk1; ++c)
#pragma unroll
            for (int turn = 0; turn < TURNS; ++turn) {
                Held b;
                load_base(b, turn, c * P_COLS);
#pragma unroll
                for (int k = 0; k < ROWS; ++k) {
                    float2 v[4] = {};
                    finish(b.u[k], v, turn * ROWS + k, c * P_COLS, true);
                }
            }
    }

    __device__ __forceinline__ void run()
    {
        if (tid == 0) {
            for (int i = 0; i < p.stages; ++i) {
                ptx::mbar_init(&full[i], P_LOADERS);
                ptx::mbar_init(&empty[i], 1);
            }
            ptx::mbar_init(done, 1);
            for (int i = 0; i < 2; ++i) {
                ptx::mbar_init(&w2_full[i], P_LOADERS);
                ptx::mbar_init(&d_full[i], 1);
                ptx::mbar_init(&d_empty[i], P_WARPS);
            }
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
        const uint32_t tmem = *slot, d2 = tmem + MOST_RANK;
        ptx::grid_dependency_wait();
        piece = p.plan.tiles[blockIdx.x / p.splits];  // the same for the whole cluster
        e = piece.adapter;
        const int chunks = p.out ? (p.to + P_COLS - 1) / P_COLS : 0;
        const int chunk0 = static_cast<int>(static_cast<int64_t>(rank_in) * chunks / p.splits), chunk1 = static_cast<int>(static_cast<int64_t>(rank_in + 1) * chunks / p.splits);
        if (piece.rows > 0) {
            if (warp < P_WARPS) make_rows();
            if (e < p.adapters)
                with(tmem, d2, chunk0, chunk1);
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

    __device__ __forceinline__ void with(uint32_t tmem, uint32_t d2, int chunk0, int chunk1)
    {
        const int steps = (p.from + P_STEP - 1) / P_STEP;
        const int s0 = static_cast<int>(static_cast<int64_t>(rank_in) * steps / p.splits), s1 = static_cast<int>(static_cast<int64_t>(rank_in + 1) * steps / p.splits);
        bool ok = true;
        if (warp < P_WARPS) {
            const __nv_bfloat16* rows[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (tid >> 3) + 32 * i;
                rows[i] = p.in + p.plan.order[piece.first + (row < piece.rows ? row : 0)] * p.in_stride + 8 * (tid & 7);
            }
            if (VEC) make_places();
            for (int f = s0; f < s1; ++f) {
                const int it = f - s0, at = it % p.stages;
                if (!wait(&empty[at], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, ok)) break;
                load_stage(mem + at * s.stage(), f * P_STEP, rows);
                arrive(&full[at]);
            }
            clear_pad(w2_buf(0));
            if (chunk0 < chunk1) load_w2(w2_buf(0), chunk0 * P_COLS);
            arrive(&w2_full[0]);
        } else {
            for (int f = s0; f < s1; ++f) {
                const int it = f - s0, at = it % p.stages;
                wait(&full[at], static_cast<uint32_t>(it / p.stages) & 1u, ok);
                ok = __all_sync(0xffffffffu, ok);  // what follows is the whole warp's
                if (!ok) break;
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
                const uint32_t a = ptx::smem_addr(mem + at * s.stage()), b = a + TILE * P_STEP * 2;
                ptx::mma_bf16_elect_x4(tmem, ptx::sw128_kmajor_desc(a), TRANS ? ptx::plain_mnmajor_desc(b, 128, W1_COLUMN) : ptx::sw128_kmajor_desc(b),
                                       32 / 16, (TRANS ? 256 : 32) / 16, TRANS ? ptx::idesc_bf16_f32_bmn(TILE, s.rp) : ptx::idesc_bf16_f32(TILE, s.rp), it > 0);
                ptx::mma_commit_elect(&empty[at]);
            }
            ptx::mma_commit_elect(done);
        }
        __syncwarp();
        wait(done, 0, ok);
        __syncwarp();
        // The ring is free: the sums, and w2's second chunk.
        float* sums = reinterpret_cast<float*>(mem);
        if (warp < 4) {
            ptx::tc_fence_after();
            const int row = 32 * warp + lane;
            for (int c = 0; c < s.rp; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c, v);
                ptx::tmem_ld_wait();
                const uint32_t at = ptx::smem_addr(sums + row * s.pitch() + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) ptx::st_shared_v4(at + 16 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            ptx::tc_fence_before();
        }
        if (p.splits > 1)
            ptx::cluster_sync();
        else
            __syncthreads();
        if (warp < P_WARPS) {
            clear_pad(w2_buf(1));
            if (chunk0 + 1 < chunk1) load_w2(w2_buf(1), (chunk0 + 1) * P_COLS);
            arrive(&w2_full[1]);
        }
        const float scale = p.scale ? __ldg(p.scale + e) : 1.f;
        switch (p.splits) {
            case 1: join<1>(sums, scale); break;
            case 2: join<2>(sums, scale); break;
            case 4: join<4>(sums, scale); break;
            default: join<8>(sums, scale); break;
        }
        if (p.splits > 1)
            ptx::cluster_sync();
        else
            __syncthreads();
        const int n = chunk1 - chunk0;
        if (warp == P_WARPS) {
            ptx::fence_proxy_async_smem();
            const uint32_t a = ptx::smem_addr(parts());
            for (int j = 0; j < n; ++j) {
                const int b = j & 1;
                const uint32_t phase = static_cast<uint32_t>(j >> 1) & 1u;
                wait(&w2_full[b], phase, ok);
                wait(&d_empty[b], phase ^ 1u, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_after();
                const uint32_t w = ptx::smem_addr(w2_buf(b));
                for (int k = 0; k < s.rp / 16; ++k)  // the three parts of 16 of mid's columns
                    ptx::mma_bf16_elect_x3(d2 + P_COLS * b, ptx::plain_kmajor_desc(a + k * 4096, 2048, 128),
                                           TRANS ? ptx::plain_mnmajor_desc(w + k * 2304, 1152, 144) : ptx::plain_kmajor_desc(w + k * 2304, 1152, 144),
                                           s.rp / 8 * (2048 / 16), TRANS ? ptx::idesc_bf16_f32_bmn(TILE, P_COLS) : ptx::idesc_bf16_f32(TILE, P_COLS), k > 0);
                ptx::mma_commit_elect(&d_full[b]);
            }
        } else if (n > 0) {
            // base a turn ahead, in two sets of registers by turns (a copy between them would wait for what is on its way)
            Held held[2];
            load_base(held[0], 0, chunk0 * P_COLS);
            for (int j0 = 0; j0 < n; j0 += 2 / TURNS)
#pragma unroll
                for (int jj = 0; jj < 2 / TURNS; ++jj) {
                    const int j = j0 + jj;
                    if (j >= n) break;
                    const int b = j & 1, c0 = (chunk0 + j) * P_COLS;
                    if (TURNS == 2 || j + 1 < n) load_base(held[TURNS == 2 ? 1 : (jj + 1) & 1], TURNS - 1, TURNS == 2 ? c0 : c0 + P_COLS);
                    wait(&d_full[b], static_cast<uint32_t>(j >> 1) & 1u, ok);
                    __syncwarp();
                    ptx::tc_fence_after();
                    uint32_t v[2][16];
                    const uint32_t at = d2 + P_COLS * b + 32 * (warp >> 2) + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
                    ptx::tmem_ld_16x256b_x4(at, v[0]);
                    ptx::tmem_ld_16x256b_x4(at + (16u << 16), v[1]);
                    if (j + 2 < n) {
                        load_w2(w2_buf(b), c0 + 2 * P_COLS);
                        arrive(&w2_full[b]);
                    }
                    ptx::tmem_ld_wait();
                    ptx::tc_fence_before();
                    if (lane == 0) ptx::mbar_arrive(&d_empty[b]);
#pragma unroll
                    for (int turn = 0; turn < TURNS; ++turn) {
                        if (turn == 1 && j + 1 < n) load_base(held[0], 0, c0 + P_COLS);
#pragma unroll
                        for (int k = 0; k < ROWS; ++k) {
                            const int i = turn * ROWS + k;
                            float2 f[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g) f[g] = make_float2(__uint_as_float(v[i >> 1][4 * g + 2 * (i & 1)]), __uint_as_float(v[i >> 1][4 * g + 2 * (i & 1) + 1]));
                            finish(held[TURNS == 1 ? jj & 1 : turn].u[k], f, i, c0, ok);
                        }
                    }
                }
        }
        __syncwarp();
        ptx::cp_async_wait_all();
        if (!ok && lane == 0 && p.status) atomicMax(p.status, 6u);
    }
};

template <bool TRANS, bool VEC, typename TB, typename TO>
__global__ void __launch_bounds__(P_THREADS, 2) pass_tiles(const __grid_constant__ PassParams p)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    Pass<TRANS, VEC, TB, TO> pass(p, raw);
    pass.run();
}

template <typename K>
int start_pass(K kernel, const PassParams& p, std::atomic<uint64_t>& done, cudaStream_t stream)
{
    const int bytes = PassSmem(p.rank, p.stages).bytes();
    if (!mx::allow_smem(kernel, 227 * 1024, done)) return CONV2D_ERR_CUDA;
    const int64_t grid = static_cast<int64_t>(p.plan.n_tiles) * p.splits;
    if (grid > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    return mx::launch(kernel, grid, P_THREADS, bytes, stream, p.splits, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

template <bool TRANS, bool VEC, typename TB, typename TO>
int start_pass_as(const PassParams& p, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return start_pass(pass_tiles<TRANS, VEC, TB, TO>, p, done, stream);
}

template <bool TRANS, bool VEC>
int start_pass_by_types(const PassParams& p, int32_t base, int32_t out, cudaStream_t stream)
{
    using B = __nv_bfloat16;
    if (base == CONV2D_OUT_BF16)
        return out == CONV2D_OUT_BF16 ? start_pass_as<TRANS, VEC, B, B>(p, stream) : start_pass_as<TRANS, VEC, B, float>(p, stream);
    return out == CONV2D_OUT_BF16 ? start_pass_as<TRANS, VEC, float, B>(p, stream) : start_pass_as<TRANS, VEC, float, float>(p, stream);
}

}  // namespace ad
}  // namespace sgb
