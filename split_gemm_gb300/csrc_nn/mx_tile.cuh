// Product of microscaled 4-bit matrices on one CTA's tensor core, with the sum
// split over a cluster: for results of few tiles, where a long sum or the
// reading of a weight has to be spread over the SMs.
//
// A tile is 128 rows of one operand (P) by BN rows of the other (Q); the
// accumulator has P's rows in its lanes.  For many rows of y, P is a and Q is b.
// For few (SWAP), P is b, the weight: its rows fill the 128 lanes whatever the
// number of rows of y, and consecutive lanes are consecutive elements of a row of y.
//
// The reduction runs in stages of 256 elements (128 bytes of a row): one TMA box
// for each operand (128-byte swizzle), and the stage's scales, which lie in memory as 512-byte tiles of
// 128 rows x 4 blocks, by bulk copies.  tcgen05.cp spreads a scale tile over 4
// columns of tensor memory; every ring slot has columns of its own, so a slot's
// scales are overwritten only after the MMAs that read them have completed.
// Four MMAs of 64 elements make a stage.
//
// CTA r of a cluster of S takes the stages [r*T/S, (r+1)*T/S).  The partial tiles
// meet in shared memory: each CTA sums 128/S rows of P over the cluster, always
// from CTA 0 to CTA S-1, so the result does not depend on timing and needs no
// workspace and no atomics.
//
// Warps 0..3: accumulator to shared memory; warp 4: copies; warp 5: MMAs.  All
// six write the result.  Every wait is bounded: on running out the status word is set and
// the CTA goes through its remaining barriers without waiting or storing.
//
// Measured: one token, 1 x 16384 x 4096 to bf16, 8.0 us, 4.5 TB/s of weight; 1 x 65536 x 8192, 54 us, 5.3 TB/s.  The MMAs do not
// bind there: a stage's take 0.18 us however few rows there are, but an SM has 16 to 32 stages to a tile, 3 us of those 8, and in the
// second case the tensor pipe is at 4%.  What does was not measured; a CTA takes one tile and fills an SM, so that each tile pays for its
// barriers, an empty ring and a drain with nothing beside it, and 128 tiles leave 24 SMs idle.  1024 x 256 x 12544 to fp32, 9.5 us, bound by what
// an SM takes from L2 and by start and join.
#pragma once

#include <cuda.h>

#include "mx_common.cuh"
#include "mx_ptx.cuh"

namespace sgb {
namespace mx {

constexpr int T_THREADS = 192;
constexpr int T_ROWS = 128;
constexpr int T_STAGE_BYTES_ROW = 128;           // of a row, in a stage
constexpr int T_STAGE_BLOCKS = 8;                // blocks of 32 in a stage
constexpr uint64_t T_WAIT_NS = 1000000000ull;

struct TileParams {
    const uint8_t *p_scales, *q_scales;
    const float* bias;
    void* y;
    uint32_t* status;
    int64_t ldy;
    int p_rows, q_rows;      // extents of the operands
    int blocks, btiles;      // of 32, and scale tiles, along the reduction
    int stages;              // T
    int q_tiles, splits;     // splits <= T, a power of two
    int relu;
    int vec_y;               // rows of y are whole groups of four elements
};

template <int BN, bool SWAP>
struct TileConfig {
    static constexpr int P_BYTES = T_ROWS * T_STAGE_BYTES_ROW;
    static constexpr int Q_BYTES = BN * T_STAGE_BYTES_ROW;
    static_assert(BN <= 128, "one scale tile along Q's rows");
    static constexpr int STAGE = P_BYTES + Q_BYTES + 4 * TILE_BYTES;  // with two scale tiles of each
    static constexpr int RING_MAX = 200 * 1024;
    static constexpr int STAGES = RING_MAX / STAGE > 8 ? 8 : RING_MAX / STAGE;
    static constexpr int SF_COLS = 16;                            // tensor-memory columns of a slot's scales
    static constexpr int COLS_USED = (BN < 32 ? 32 : BN) + STAGES * SF_COLS;
    static constexpr uint32_t TMEM_COLS = COLS_USED <= 128 ? 128 : (COLS_USED <= 256 ? 256 : 512);
    static_assert(COLS_USED <= 512, "tensor memory");
    // The staged tile, in y's order: rows of BN (SWAP: of 128) words and 4 more, so that 16-byte accesses of
    // neighbouring rows fall into different banks.
    static constexpr int PITCH = (SWAP ? T_ROWS : BN) + 4;
    static constexpr int STAGED = (SWAP ? BN : T_ROWS) * PITCH * 4;
    static constexpr int RING = STAGES * STAGE > STAGED ? STAGES * STAGE : STAGED;
    static constexpr int SMEM = RING + 1024 + 256;                // + alignment, barriers
};

// The sum of four values over the S CTAs of the cluster, in their order; the loads are on their way together.
template <int S>
__device__ __forceinline__ float4 joined4(const float* at)
{
    if constexpr (S == 1) {
        return *reinterpret_cast<const float4*>(at);
    } else {
        float4 v[S];
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] = ptx::ld_cluster_v4(ptx::mapa_shared(ptx::smem_addr(at), k));
#pragma unroll
        for (int k = 1; k < S; ++k) {
            v[0].x += v[k].x;
            v[0].y += v[k].y;
            v[0].z += v[k].z;
            v[0].w += v[k].w;
        }
        return v[0];
    }
}

// Joins and writes this CTA's share of the tile, 128/S of P's rows, four elements of a row of y to a thread.
template <int S, int BN, bool SWAP, typename T>
__device__ __forceinline__ void write_share(float* staged, int rank, int p0, int q0, int q_valid, const TileParams& p)
{
    constexpr int SHARE = T_ROWS / S, PITCH = TileConfig<BN, SWAP>::PITCH;
    constexpr int WIDTH = SWAP ? SHARE : BN;  // of a row of the share
    static_assert(T_THREADS % (WIDTH / 4) == 0, "a thread keeps its columns");
    // A thread keeps its four columns and goes down the rows.
    const int r0 = rank * SHARE;
    const int height = SWAP ? q_valid : SHARE;
    const int rows = SWAP ? p.q_rows : p.p_rows, cols = SWAP ? p.p_rows : p.q_rows;  // of y
    // rows and columns of the staged tile, and where they are in y
    const int first_row = SWAP ? 0 : r0, first_col = SWAP ? r0 : 0, y_row = SWAP ? q0 : p0, y_col = SWAP ? p0 : q0;
    const int left = rows - (y_row + first_row), n_rows = left < height ? left : height;
    T* y = static_cast<T*>(p.y);
    constexpr int LANES = WIDTH / 4;
    const int c = first_col + threadIdx.x % LANES * 4, col = y_col + c;
    if (col < cols) {
        float bias[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < cols) bias[i] = __ldg(p.bias + col + i);
#pragma unroll 2
        for (int r = threadIdx.x / LANES; r < n_rows; r += T_THREADS / LANES) {
            float* at = staged + (first_row + r) * PITCH + c;
            const float4 s = joined4<S>(at);
            float v[4] = {s.x + bias[0], s.y + bias[1], s.z + bias[2], s.w + bias[3]};
            if (p.relu)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v[i] < 0.f) v[i] = 0.f;
            T* out = y + static_cast<int64_t>(y_row + first_row + r) * p.ldy + col;
            if (!p.vec_y) {
                *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
            } else if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
        }
    }
    if (p.vec_y) return;
    // Rows of y that begin anywhere: the finished values went back to where they lay (no other CTA reads this share), and
    // leave in 16-byte stores from the first aligned place of each row on, the few before and after one by one.
    __syncthreads();
    constexpr int EV = 16 / sizeof(T), ROW_LANES = WIDTH / EV;
    const int lane = threadIdx.x % ROW_LANES;
    const int valid = cols - (y_col + first_col) < WIDTH ? cols - (y_col + first_col) : WIDTH;
    for (int r = threadIdx.x / ROW_LANES; r < n_rows; r += T_THREADS / ROW_LANES) {
        const float* from = staged + (first_row + r) * PITCH + first_col;
        const int64_t g = static_cast<int64_t>(y_row + first_row + r) * p.ldy + y_col + first_col;  // y is aligned to 16 bytes
        const int head = static_cast<int>(-g & (EV - 1));
        const int at = head + lane * EV;
        if (at + EV <= valid) {
            alignas(16) T v[EV];
#pragma unroll
            for (int i = 0; i < EV; ++i) from_float(v[i], from[at + i]);
            *reinterpret_cast<uint4*>(y + g + at) = *reinterpret_cast<const uint4*>(v);
        }
        for (int e = lane; e < head && e < valid; e += ROW_LANES) from_float(y[g + e], from[e]);
        const int tail = valid > head ? head + (valid - head) / EV * EV : valid;
        for (int e = tail + lane; e < valid; e += ROW_LANES) from_float(y[g + e], from[e]);
    }
}

template <int BN, bool SWAP, typename T>
__global__ void __launch_bounds__(T_THREADS, 1) tile_kernel(const __grid_constant__ CUtensorMap tm_p,
                                                         const __grid_constant__ CUtensorMap tm_q, const TileParams p)
{
    using C = TileConfig<BN, SWAP>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + C::RING);
    uint64_t* empty = full + C::STAGES;
    uint64_t* done = empty + C::STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % p.splits, tile = blockIdx.x / p.splits;
    const int p0 = tile / p.q_tiles * T_ROWS, q0 = tile % p.q_tiles * BN;
    const int s0 = static_cast<int>(static_cast<int64_t>(rank) * p.stages / p.splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.stages / p.splits);

    if (threadIdx.x < 2) ptx::prefetch_tensormap(threadIdx.x ? &tm_q : &tm_p);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0u;
        ptx::mbar_init_fence();
    }
    if (warp == 5) {
        ptx::tmem_alloc(tmem_slot, C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t acc = *tmem_slot, sf = acc + (BN < 32 ? 32 : BN);
    ptx::grid_dependency_wait();

    if (warp == 4 && lane == 0) {
        int it = 0;
        for (int s = s0; s < s1; ++s, ++it) {
            const int slot = it % C::STAGES;
            if (!ptx::mbar_wait(&empty[slot], (static_cast<uint32_t>(it / C::STAGES) & 1u) ^ 1u, T_WAIT_NS)) {
                *abort_flag = 1u;
                break;
            }
            uint8_t* st = ring + slot * C::STAGE;
            uint8_t* sfs = st + C::P_BYTES + C::Q_BYTES;
            const int left = p.btiles - 2 * s;
            const uint32_t sbytes = static_cast<uint32_t>(left < 2 ? left : 2) * TILE_BYTES;
            ptx::mbar_arrive_expect_tx(&full[slot], C::P_BYTES + C::Q_BYTES + 2 * sbytes);
            ptx::tma_load_2d(st, &tm_p, &full[slot], s * T_STAGE_BYTES_ROW, p0);
            ptx::tma_load_2d(st + C::P_BYTES, &tm_q, &full[slot], s * T_STAGE_BYTES_ROW, q0);
            ptx::bulk_load(sfs, p.p_scales + (static_cast<int64_t>(p0 / 128) * p.btiles + 2 * s) * TILE_BYTES, sbytes, &full[slot]);
            ptx::bulk_load(sfs + 2 * TILE_BYTES, p.q_scales + (static_cast<int64_t>(q0 / 128) * p.btiles + 2 * s) * TILE_BYTES, sbytes,
                           &full[slot]);
        }
        // copies in flight land before the CTA ends
        for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
            if (!ptx::mbar_wait(&full[i % C::STAGES], static_cast<uint32_t>(i / C::STAGES) & 1u, T_WAIT_NS)) *abort_flag = 1u;
    } else if (warp == 5) {  // the whole warp, so that operands stay uniform; one lane issues
        int it = 0;
        for (int s = s0; s < s1; ++s, ++it) {
            const int slot = it % C::STAGES;
            if (!ptx::mbar_wait_spin(&full[slot], static_cast<uint32_t>(it / C::STAGES) & 1u, T_WAIT_NS)) {
                *abort_flag = 1u;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t st = ptx::smem_addr(ring + slot * C::STAGE);
            const int left = p.blocks - s * T_STAGE_BLOCKS;
            ptx::mma_mxf4_stage(acc, ptx::sw128_kmajor_desc(st), ptx::sw128_kmajor_desc(st + C::P_BYTES),
                                ptx::plain_kmajor_desc(st + C::P_BYTES + C::Q_BYTES, 128, 128), sf + slot * C::SF_COLS, q0 % TILE_ROWS / 32,
                                ptx::idesc_mxf4(T_ROWS, BN, 0), ptx::idesc_mxf4(T_ROWS, BN, 2), it > 0,
                                left >= T_STAGE_BLOCKS ? 4 : (left + 1) / 2);
            ptx::mma_commit_elect(&empty[slot]);
        }
        ptx::mma_commit_elect(done);
    }
    __syncwarp();

    // The accumulator to shared memory (the ring is free once all MMAs are done).
    float* staged = reinterpret_cast<float*>(ring);
    const int q_left = p.q_rows - q0;
    const int q_valid = q_left < BN ? q_left : BN;
    const bool ok = ptx::mbar_wait(done, 0, 2 * T_WAIT_NS);
    if (!ok) *abort_flag = 1u;
    __syncthreads();  // also: the copies' thread has seen its last copy land
    if (warp < 4) {
        ptx::tc_fence_after();
        constexpr int STEP = BN < 64 ? 16 : 64;  // columns on their way at once
        const int row = warp * 32 + lane;
        for (int c = 0; c < q_valid; c += STEP) {
            uint32_t v[STEP / 16][16];
#pragma unroll
            for (int k = 0; k < STEP / 16; ++k) ptx::tmem_ld_32x32b_x16(acc + (static_cast<uint32_t>(warp * 32) << 16) + c + 16 * k, v[k]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < STEP / 16; ++k) {
                if constexpr (SWAP) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) staged[(c + 16 * k + i) * C::PITCH + row] = __uint_as_float(v[k][i]);
                } else {
                    const uint32_t at = ptx::smem_addr(staged + row * C::PITCH + c + 16 * k);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ptx::st_shared_v4(at + 16 * i, v[k][4 * i], v[k][4 * i + 1], v[k][4 * i + 2], v[k][4 * i + 3]);
                }
            }
        }
        ptx::tc_fence_before();
    }
    const bool failed = *abort_flag != 0u;
    if (p.splits > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    if (failed) {
        if (threadIdx.x == 0 && p.status) atomicMax(p.status, 6u);
    } else {
        switch (p.splits) {
            case 1: write_share<1, BN, SWAP, T>(staged, 0, p0, q0, q_valid, p); break;
            case 2: write_share<2, BN, SWAP, T>(staged, rank, p0, q0, q_valid, p); break;
            case 4: write_share<4, BN, SWAP, T>(staged, rank, p0, q0, q_valid, p); break;
            default: write_share<8, BN, SWAP, T>(staged, rank, p0, q0, q_valid, p); break;
        }
    }
    if (p.splits > 1) ptx::cluster_sync();  // the others have read this CTA's part
    __syncthreads();
    if (warp == 5) ptx::tmem_dealloc(acc, C::TMEM_COLS);
}

}  // namespace mx
}  // namespace sgb
