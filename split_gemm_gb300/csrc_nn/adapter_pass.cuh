// One direction through the adapters, in [rows][from] -> mid [rows][rank] -> out [rows][to], by tiles of up to 128 rows of one adapter:
//
//   mid = scale * in w1^T,  out = act(base + mid w2^T)
//
// Forward w1 is a[e] and w2 is b[e], both K-major operands; backward (TRANS) w1 is b[e]^T and w2 a[e]^T, both MN-major.
//
// in, base and out each pass once over HBM and bind it: with rank r the matrix units have 2r flops to some 4 bytes.  A cluster
// of S CTAs shares a tile: each takes a part of `from` for the first product, 128/S rows of the join and a part of `to` for the
// second, so that few tiles fill the SMs and the smaller the parts, the more tiles are at different phases at once on an SM (two CTAs stay there up
// to rank 64).  mid never leaves the chip but for the copy that the gradients need.
//
// First product: rows of `in` are gathered by the plan's order with cp.async into core matrices of 8 rows x 16 bytes (no
// swizzle); a quarter warp copies one 16-byte column of 8 rows, which is conflict-free in shared memory, a warp 64 bytes of each row.  128 x rank
// x 64 a stage.  The sums over the parts meet in shared memory as fp32, are joined in the CTAs' order and cut into three bf16 parts that
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

    // Columns f0 .. f0+63 of the tile's rows and of w1.
    __device__ __forceinline__ void load_stage(uint8_t* st, int f0, const __nv_bfloat16* const (&rows)[2]) const
    {
        const uint32_t at = ptx::smem_addr(st);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (lane & 7) + 8 * warp + 64 * (i & 1), c8 = (lane >> 3) + 4 * (i >> 1);
            if (row < piece.rows) copy8(at + (row & 7) * 16 + (row >> 3) * 128 + c8 * 2048, rows[i & 1] + f0 + 8 * c8, p.from - f0 - 8 * c8);
        }
        const uint32_t w_at = at + TILE * P_STEP * 2;
        const int64_t size = static_cast<int64_t>(p.rank) * p.from;
        const __nv_bfloat16* w = p.w1 + e * size;
        if constexpr (!TRANS) {
            for (int i = tid; i < s.rp * 8; i += P_LOADERS) {  // rows of 8 16-byte columns
                const int group = i >> 5, groups = s.rp >> 3, half = group >= groups;
                const int r = (i & 7) + 8 * (group - half * groups), c8 = ((i >> 3) & 3) + 4 * half;
                if (r < p.rank) copy8(w_at + (r & 7) * 16 + (r >> 3) * 128 + c8 * (s.rp * 16), w + static_cast<int64_t>(r) * p.from + f0 + 8 * c8, p.from - f0 - 8 * c8);
            }
        } else {
            for (int i = tid; i < s.rp * 8; i += P_LOADERS) {  // 64 rows of rp/8 16-byte columns
                const int k = (i >> 1) & 63, n8 = 2 * (i >> 7) + (i & 1);
                const int left = f0 + k < p.from ? p.rank - 8 * n8 : 0;
                copy8(w_at + (k & 7) * 16 + n8 * 1024 + (k >> 3) * 128, w + static_cast<int64_t>(f0 + k) * p.rank + 8 * n8, left);
            }
        }
    }

    // w2's 64 columns from c0 on: column c of 32 becomes row 8((c>>1)&3) + 2(c>>3) + (c&1) of the operand.
    __device__ __forceinline__ void load_w2(uint8_t* buf, int c0) const
    {
        const uint32_t at = ptx::smem_addr(buf);
        const int64_t size = static_cast<int64_t>(p.rank) * p.to;
        const __nv_bfloat16* w = p.w2 + e * size;
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

    // This CTA's rows of the sums over the cluster: scaled, to mid, and in three parts to every CTA.
    template <int S>
    __device__ __forceinline__ void join(const float* sums, float scale) const
    {
        constexpr int SHARE = TILE / S;
        const int quads = s.rp >> 2;
        for (int i = tid; i < SHARE * quads; i += P_THREADS) {
            const int row = rank_in * SHARE + i % SHARE, r = 4 * (i / SHARE);
            const float* at = sums + row * s.pitch() + r;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (row < piece.rows) {
                if constexpr (S == 1) {
                    *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(at);
                } else {
                    float4 u[S];
#pragma unroll
                    for (int k = 0; k < S; ++k) u[k] = ptx::ld_cluster_v4(ptx::mapa_shared(ptx::smem_addr(at), k));
#pragma unroll
                    for (int k = 0; k < S; ++k) {
                        v[0] += u[k].x;
                        v[1] += u[k].y;
                        v[2] += u[k].z;
                        v[3] += u[k].w;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = r + j < p.rank ? v[j] * scale : 0.f;
                if (p.mid) {
                    float* mid = p.mid + static_cast<int64_t>(p.plan.order[piece.first + row]) * p.rank + r;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (r + j < p.rank) mid[j] = v[j];
                }
            }
            uint32_t part[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split3(v[j], part[0][j], part[1][j], part[2][j]);
            const uint32_t to = ptx::smem_addr(parts()) + (row & 7) * 16 + (row >> 3) * 128 + (r & 4) * 2;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const uint32_t dst = to + ((q * s.rp + r) >> 3) * 2048;
                const uint32_t lo = part[q][0] | part[q][1] << 16, hi = part[q][2] | part[q][3] << 16;
                if constexpr (S == 1) {
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(lo), "r"(hi) : "memory");
                } else {
#pragma unroll
                    for (int k = 0; k < S; ++k) ptx::st_cluster_v2(ptx::mapa_shared(dst, k), lo, hi);
                }
            }
        }
        ptx::fence_proxy_async_all();
    }

    // 8 elements of a row from column c on, of which `left` exist.
    template <typename T>
    struct Eight {
        static constexpr int N = sizeof(T) / 2;
        uint4 u[N];
        __device__ __forceinline__ void load(const T* row, int left)
        {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = make_uint4(0, 0, 0, 0);
            if (left <= 0) return;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < N; ++i) u[i] = __ldcs(reinterpret_cast<const uint4*>(row) + i);
            } else {
                T* v = reinterpret_cast<T*>(u);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < left) v[i] = row[i];
            }
        }
        __device__ __forceinline__ float at(int i) const
        {
            if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(u)[i];
            const uint32_t w = reinterpret_cast<const uint32_t*>(u)[i / 2];
            return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
        }
    };
    __device__ __forceinline__ static void store8(TO* row, const float (&v)[8], int left)
    {
        if (left <= 0) return;
        if constexpr (VEC) {
            if constexpr (sizeof(TO) == 4) {
                __stcs(reinterpret_cast<float4*>(row), make_float4(v[0], v[1], v[2], v[3]));
                __stcs(reinterpret_cast<float4*>(row) + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                __stcs(reinterpret_cast<uint4*>(row), make_uint4(o[0], o[1], o[2], o[3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) mx::from_float(row[i], v[i]);
        }
    }

    // A thread's rows of a tile (of its warp's 32 lanes, every 8th) and their elements of a chunk of 64 columns: 8 of the warp's 32.
    int tokens[4];
    __device__ __forceinline__ int row_of(int i) const { return 32 * (warp & 3) + (lane >> 2) + 8 * i; }
    __device__ __forceinline__ int col_of(int c0) const { return c0 + 32 * (warp >> 2) + 8 * (lane & 3); }
    __device__ __forceinline__ void load_base(Eight<TB> (&b)[4], int c0) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[i].load(static_cast<const TB*>(p.base) + tokens[i] * p.base_stride + col_of(c0), p.base && row_of(i) < piece.rows ? p.to - col_of(c0) : 0);
    }
    __device__ __forceinline__ void finish(const Eight<TB>& b, float (&v)[8], int i, int c0, bool live) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] += b.at(j);
            if (p.relu && v[j] < 0.f) v[j] = 0.f;
        }
        store8(static_cast<TO*>(p.out) + tokens[i] * p.out_stride + col_of(c0), v, live && row_of(i) < piece.rows ? p.to - col_of(c0) : 0);
    }

    // Rows without an adapter: out = act(base), mid = 0.
    __device__ __forceinline__ void without(int chunk0, int chunk1) const
    {
        if (p.mid && rank_in == 0)
            for (int i = tid; i < piece.rows * p.rank; i += P_THREADS)
                p.mid[static_cast<int64_t>(p.plan.order[piece.first + i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (!p.out || warp >= P_WARPS) return;
        for (int c = chunk0; c < chunk1; ++c) {
            Eight<TB> b[4];
            load_base(b, c * P_COLS);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8] = {};
                finish(b[i], v, i, c * P_COLS, true);
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
#pragma unroll
            for (int i = 0; i < 4; ++i) tokens[i] = p.plan.order[piece.first + (row_of(i) < piece.rows ? row_of(i) : 0)];
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
            const __nv_bfloat16* rows[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = (lane & 7) + 8 * warp + 64 * i;
                rows[i] = p.in + p.plan.order[piece.first + (row < piece.rows ? row : 0)] * p.in_stride;
            }
            for (int f = s0; f < s1; ++f) {
                const int it = f - s0, at = it % p.stages;
                if (!wait(&empty[at], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, ok)) break;
                load_stage(mem + at * s.stage(), f * P_STEP, rows);
                arrive(&full[at]);
            }
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
#pragma unroll
                for (int k = 0; k < P_STEP / 16; ++k)
                    ptx::mma_bf16_elect(tmem, ptx::plain_kmajor_desc(a + k * 4096, 2048, 128),
                                        TRANS ? ptx::plain_mnmajor_desc(b + k * 256, 128, 1024) : ptx::plain_kmajor_desc(b + k * 2 * s.rp * 16, s.rp * 16, 128),
                                        TRANS ? ptx::idesc_bf16_f32_bmn(TILE, s.rp) : ptx::idesc_bf16_f32(TILE, s.rp), it > 0 || k > 0);
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
                for (int q = 0; q < 3; ++q)
                    for (int k = 0; k < s.rp / 16; ++k)
                        ptx::mma_bf16_elect(d2 + P_COLS * b, ptx::plain_kmajor_desc(a + ((q * s.rp >> 3) + 2 * k) * 2048, 2048, 128),
                                            TRANS ? ptx::plain_mnmajor_desc(w + k * 2304, 1152, 144) : ptx::plain_kmajor_desc(w + k * 2304, 1152, 144),
                                            TRANS ? ptx::idesc_bf16_f32_bmn(TILE, P_COLS) : ptx::idesc_bf16_f32(TILE, P_COLS), q > 0 || k > 0);
                ptx::mma_commit_elect(&d_full[b]);
            }
        } else if (n > 0) {
            Eight<TB> now[4], next[4];
            load_base(now, chunk0 * P_COLS);
            for (int j = 0; j < n; ++j) {
                const int b = j & 1, c0 = (chunk0 + j) * P_COLS;
                if (j + 1 < n) load_base(next, c0 + P_COLS);
                wait(&d_full[b], static_cast<uint32_t>(j >> 1) & 1u, ok);
                __syncwarp();
                ptx::tc_fence_after();
                uint32_t v[2][16];
                const uint32_t at = d2 + P_COLS * b + 32 * (warp >> 2) + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
                ptx::tmem_ld_16x256b_x4(at, v[0]);
                ptx::tmem_ld_16x256b_x4(at + (16u << 16), v[1]);
                if (j + 2 < n) load_w2(w2_buf(b), c0 + 2 * P_COLS);
                if (j + 2 < n) arrive(&w2_full[b]);
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                if (lane == 0) ptx::mbar_arrive(&d_empty[b]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[i >> 1][4 * (k >> 1) + 2 * (i & 1) + (k & 1)]);
                    finish(now[i], f, i, c0, ok);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = next[i];
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
