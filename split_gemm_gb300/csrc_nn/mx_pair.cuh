// Product of microscaled 4-bit matrices on CTA pairs: 256 x 256 tiles, persistent.
//
// What bounds it: at 4-bit rates a 256 x 256 x 64 MMA of a pair takes 128 cycles, in which each SM needs 8 KB
// of operands; the largest tile that tensor memory holds (256 fp32 columns beside the scales) is therefore taken
// even though a second accumulator does not fit.  Its place is taken by a short drain: eight warps read the
// accumulator into registers (about 128 columns each, a few hundred cycles), hand it back to the MMAs of the next tile and
// write y while those run.
//
// A stage is 256 reduction elements.  Each CTA loads its 128 rows of a, its half of b's 256 rows (128-byte
// swizzle), the scales of its rows of a and of all the tile's rows of b (512-byte scale tiles as a tensor of
// 128 words x blocks/4 x rows/128, so that what lies beyond reads as zero).  Both CTAs' loads count on the leader's
// barrier; the leader's commit frees the slot in both.  Scales have tensor-memory columns of their own for every
// slot, so a slot's scales are overwritten only after the MMAs that read them have completed.
//
// Warps: 0 copies (one thread), 1 MMAs (one thread of the leader), 2..9 accumulator to y.  y goes out by TMA
// stores of 32-row boxes, or element by element where its rows are not a multiple of 16 bytes.
//
// Measured: 8192 x 8192 x 8192 to bf16 163 us, 6.8 PFLOP/s; 1024 x 4096 x 4096 11 us.  Of the 8192 cube the MMAs alone are
// 119 us; without loads it would take 135, without stores 155, so most of the rest is the operands' way from L2.  Five stages, as four
// cost 181 us and three 215.
#pragma once

#include "mx_tile.cuh"

namespace sgb {
namespace mx {

constexpr int W_TILE = 256;
constexpr int W_BAND = 16;         // row blocks of tiles taken together
constexpr int W_ROWS = 128;        // of a, and of b, that a CTA holds
constexpr int W_STAGES = 5;
constexpr int W_AB = W_ROWS * T_STAGE_BYTES_ROW;
constexpr int W_SFA = 2 * TILE_BYTES, W_SFB = 4 * TILE_BYTES;
constexpr int W_STAGE = 2 * W_AB + W_SFA + W_SFB;      // 35 KB
constexpr int W_EPI_WARPS = 8;
constexpr int W_BOX = 32 * 128;                        // 32 rows of 128 bytes
constexpr int W_THREADS = 32 * (2 + W_EPI_WARPS);
constexpr int W_SMEM = W_STAGES * W_STAGE + W_EPI_WARPS * (W_BOX + 512) + 1024 + 256;  // + each warp's bias, alignment, barriers
constexpr int W_SF_COLS = 24;                          // of a slot: 2 x 4 for a, 2 x 8 for b
static_assert(W_TILE + W_STAGES * W_SF_COLS <= 512, "tensor memory");
static_assert(W_SMEM <= 232448 && W_STAGE % 1024 == 0, "shared memory");

struct PairParams {
    const float* bias;
    void* y;
    uint32_t* status;
    int64_t ldy;
    int m, n;
    int stages;
    int m_tiles, n_tiles;
    int relu, tma_store;
};

// Tile number to row and column block: bands of 16 row blocks, columns within a band, rows fastest, so that the
// tiles in flight share few rows and columns of the operands in L2.
__device__ __forceinline__ void tile_of(int i, const PairParams& p, int& tm, int& tn)
{
    const int band = i / (W_BAND * p.n_tiles), rest = i - band * W_BAND * p.n_tiles;
    const int rows = p.m_tiles - band * W_BAND < W_BAND ? p.m_tiles - band * W_BAND : W_BAND;
    tn = rest / rows;
    tm = band * W_BAND + rest - tn * rows;
}

template <typename T>
__global__ void __launch_bounds__(W_THREADS, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                const __grid_constant__ CUtensorMap tm_y, const PairParams p)
{
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* boxes = ring + W_STAGES * W_STAGE;
    float* biases = reinterpret_cast<float*>(boxes + W_EPI_WARPS * W_BOX);
    uint64_t* full = reinterpret_cast<uint64_t*>(biases + W_EPI_WARPS * 128);
    uint64_t* empty = full + W_STAGES;
    uint64_t* acc_full = empty + W_STAGES;
    uint64_t* acc_empty = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const int cluster = static_cast<int>(ptx::cluster_id_x()), clusters = static_cast<int>(ptx::cluster_count_x());
    const int tiles = p.m_tiles * p.n_tiles;

    if (threadIdx.x < 4) ptx::prefetch_tensormap(threadIdx.x == 0 ? &tm_a : threadIdx.x == 1 ? &tm_b : threadIdx.x == 2 ? &tm_sa : &tm_sb);
    if (threadIdx.x == 0) {
        for (int i = 0; i < W_STAGES; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(acc_full, 1);
        ptx::mbar_init(acc_empty, 2 * W_EPI_WARPS);
        *abort_flag = 0u;
        ptx::mbar_init_fence();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_slot, 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t acc = *tmem_slot, sf = acc + W_TILE;
    ptx::grid_dependency_wait();

    if (warp == 0 && lane == 0) {
        const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(full), 0);
        int it = 0;
        for (int tile = cluster; tile < tiles && !*abort_flag; tile += clusters) {
            int tm, tn;
            tile_of(tile, p, tm, tn);
            const int row_a = tm * W_TILE + static_cast<int>(rank) * W_ROWS, row_b = tn * W_TILE + static_cast<int>(rank) * W_ROWS;
            for (int s = 0; s < p.stages; ++s, ++it) {
                const int slot = it % W_STAGES;
                if (!ptx::mbar_wait(&empty[slot], (static_cast<uint32_t>(it / W_STAGES) & 1u) ^ 1u, T_WAIT_NS)) {
                    *abort_flag = 1u;
                    break;
                }
                uint8_t* st = ring + slot * W_STAGE;
                const uint32_t bar = full0 + slot * 8;
                if (rank == 0) ptx::mbar_arrive_expect_tx(&full[slot], 2 * W_STAGE);
                ptx::tma_load_2d_pair(st, &tm_a, bar, s * T_STAGE_BYTES_ROW, row_a);
                ptx::tma_load_2d_pair(st + W_AB, &tm_b, bar, s * T_STAGE_BYTES_ROW, row_b);
                ptx::tma_load_3d_pair(st + 2 * W_AB, &tm_sa, bar, 0, 2 * s, row_a / TILE_ROWS);
                ptx::tma_load_3d_pair(st + 2 * W_AB + W_SFA, &tm_sb, bar, 0, 2 * s, tn * 2);
            }
        }
        // The last use of each slot is over (its copies have landed and been read) once the leader frees it.
        for (int i = it > W_STAGES ? it - W_STAGES : 0; i < it; ++i)
            if (!ptx::mbar_wait(&empty[i % W_STAGES], static_cast<uint32_t>(i / W_STAGES) & 1u, T_WAIT_NS)) *abort_flag = 1u;
    } else if (warp == 1 && rank == 0) {  // the whole warp, so that operands stay uniform; one lane issues
        int it = 0, n = 0;
        for (int tile = cluster; tile < tiles && !*abort_flag; tile += clusters, ++n) {
            if (!ptx::mbar_wait(acc_empty, (static_cast<uint32_t>(n) & 1u) ^ 1u, T_WAIT_NS)) {
                *abort_flag = 1u;
                break;
            }
            ptx::tc_fence_after();
            for (int s = 0; s < p.stages; ++s, ++it) {
                const int slot = it % W_STAGES;
                if (!ptx::mbar_wait_spin(&full[slot], static_cast<uint32_t>(it / W_STAGES) & 1u, T_WAIT_NS)) {
                    *abort_flag = 1u;
                    break;
                }
                ptx::tc_fence_after();
                // Past the reduction's end elements and scales read as zero, so the last stage takes four MMAs too.
                const uint32_t st = ptx::smem_addr(ring + slot * W_STAGE);
                ptx::mma_mxf4_pair_stage(acc, ptx::sw128_kmajor_desc(st), ptx::sw128_kmajor_desc(st + W_AB),
                                         ptx::plain_kmajor_desc(st + 2 * W_AB, 128, 128), sf + slot * W_SF_COLS,
                                         ptx::idesc_mxf4(W_TILE, W_TILE, 0), ptx::idesc_mxf4(W_TILE, W_TILE, 2), s > 0);
                ptx::mma_commit_pair_elect(&empty[slot], 3);
            }
            ptx::mma_commit_pair_elect(acc_full, 3);
        }
    } else if (warp >= 2) {
        const int quad = warp & 3, half = (warp - 2) >> 2;  // lanes 32*quad.., columns 128*half..
        uint8_t* box = boxes + (warp - 2) * W_BOX;
        const uint32_t box_addr = ptx::smem_addr(box);
        const uint32_t release = ptx::mapa_shared(ptx::smem_addr(acc_empty), 0);
        constexpr int COLS = 128 / sizeof(T);  // of a box
        int n = 0;
        for (int tile = cluster; tile < tiles && !*abort_flag; tile += clusters, ++n) {
            int tm, tn;
            tile_of(tile, p, tm, tn);
            const int row0 = tm * W_TILE + static_cast<int>(rank) * W_ROWS + quad * 32, col0 = tn * W_TILE + half * 128;
            if (p.bias) {  // this warp's 128 columns, while the MMAs run
                __syncwarp();
                float* mine = biases + (warp - 2) * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = lane + 32 * i;
                    mine[c] = col0 + c < p.n ? __ldg(p.bias + col0 + c) : 0.f;
                }
                __syncwarp();
            }
            if (!ptx::mbar_wait(acc_full, static_cast<uint32_t>(n) & 1u, 2 * T_WAIT_NS)) {
                *abort_flag = 1u;
                break;
            }
            ptx::tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                ptx::tmem_ld_32x32b_x32(acc + (static_cast<uint32_t>(quad * 32) << 16) + half * 128 + c * 32, v[c]);
            ptx::tmem_ld_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster(release);
            if (row0 >= p.m || col0 >= p.n) continue;
            if (p.bias) {
                const float4* mine = reinterpret_cast<const float4*>(biases + (warp - 2) * 128);
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 b = mine[c * 8 + i];
                        const float2 lo = add2(make_float2(__uint_as_float(v[c][4 * i]), __uint_as_float(v[c][4 * i + 1])), make_float2(b.x, b.y));
                        const float2 hi = add2(make_float2(__uint_as_float(v[c][4 * i + 2]), __uint_as_float(v[c][4 * i + 3])), make_float2(b.z, b.w));
                        v[c][4 * i] = __float_as_uint(lo.x);
                        v[c][4 * i + 1] = __float_as_uint(lo.y);
                        v[c][4 * i + 2] = __float_as_uint(hi.x);
                        v[c][4 * i + 3] = __float_as_uint(hi.y);
                    }
            }
            if (sizeof(T) == 4 && p.relu) {  // bf16 values are clamped by pairs after rounding, which is the same
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[c][i] = ptx::relu_nan(v[c][i]);
            }
#pragma unroll
            for (int b = 0; b < 128 / COLS; ++b) {
                if (col0 + b * COLS >= p.n) break;
                // the box is free once the last store from it has been read
                if (lane == 0) ptx::bulk_wait_read_all();
                __syncwarp();
                const uint32_t at = box_addr + lane * 128;
#pragma unroll
                for (int q = 0; q < 8; ++q) {  // 16 bytes each, swizzled by the row
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (sizeof(T) == 4) {
                            w[i] = v[b][4 * q + i];
                        } else {
                            const int e = b * 64 + q * 8 + 2 * i;
                            __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1]));
                            if (p.relu) h = __hmax2_nan(h, __nv_bfloat162(__float2bfloat16_rn(0.f), __float2bfloat16_rn(0.f)));
                            w[i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    ptx::st_shared_v4(at + ((q ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                if (p.tma_store) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(&tm_y, box, col0 + b * COLS, row0);
                        ptx::bulk_commit();
                    }
                } else {
                    __syncwarp();
                    // Rows of y that begin anywhere.  fp32: the warp stores a row of the box at a time, a word to a lane.  bf16, where
                    // that would be half words: eight lanes to a row, 16-byte stores from the first aligned place on, the rest one by
                    // one.  (13567 x 10797 x 128: fp32 249 us, the other way 275; bf16 177, the other way 213; in a graph
                    // 234 and 155, with 10800 columns, which go by boxes, 103 and 75.)
                    T* y = static_cast<T*>(p.y);
                    const int c0 = col0 + b * COLS, left_c = p.n - c0, valid = left_c < COLS ? left_c : COLS;
                    if constexpr (sizeof(T) == 4) {
                        const int rows = p.m - row0 < 32 ? p.m - row0 : 32;
                        T* out = y + static_cast<int64_t>(row0) * p.ldy + c0;
#pragma unroll 8
                        for (int r = 0; r < rows; ++r, out += p.ldy)
                            if (lane < valid) out[lane] = *reinterpret_cast<const T*>(box + r * 128 + ((lane * 4) ^ ((r & 7) << 4)));
                    } else {
                        constexpr int EV = 16 / sizeof(T);
                        auto value = [&](int r, int c) {
                            return *reinterpret_cast<const T*>(box + r * 128 + ((c * static_cast<int>(sizeof(T))) ^ ((r & 7) << 4)));
                        };
                        for (int r = lane / 8; r < 32 && row0 + r < p.m; r += 4) {
                            const int64_t g = static_cast<int64_t>(row0 + r) * p.ldy + c0;  // y is aligned to 16 bytes
                            const int head = static_cast<int>(-g & (EV - 1)), at_c = head + lane % 8 * EV;
                            if (at_c + EV <= valid) {
                                alignas(16) T o[EV];
#pragma unroll
                                for (int i = 0; i < EV; ++i) o[i] = value(r, at_c + i);
                                *reinterpret_cast<uint4*>(y + g + at_c) = *reinterpret_cast<const uint4*>(o);
                            }
                            if (lane % 8 < head && lane % 8 < valid) y[g + lane % 8] = value(r, lane % 8);
                            const int tail = valid > head ? head + (valid - head) / EV * EV : valid;
                            if (tail + lane % 8 < valid) y[g + tail + lane % 8] = value(r, tail + lane % 8);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_read_all();
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // let copies in flight land before this CTA's memory goes
        const uint64_t t0 = ptx::clock64();
        while (ptx::clock64() - t0 < ptx::ns_to_cycles(1000000ull)) {
        }
        if (p.status) atomicMax(p.status, 6u);
    }
    __syncthreads();
    ptx::cluster_sync();
    if (warp == 1) ptx::tmem_dealloc_pair(acc, 512);
}

}  // namespace mx
}  // namespace sgb
