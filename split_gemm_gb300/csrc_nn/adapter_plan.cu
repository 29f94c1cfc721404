// Makes adapter plans: a stable counting sort of the rows by adapter, in three launches.
#include "adapter_plan.cuh"

#include "adapter.h"
#include "ptx.cuh"

namespace sgb {
namespace ad {

struct PlanParams {
    const int* index;
    int* w;
    PlanLayout l;
};

__device__ __forceinline__ int adapter_of(const PlanParams& p, int64_t row)
{
    const int e = __ldg(p.index + row);
    const int none = static_cast<int>(p.l.adapters);
    return static_cast<unsigned>(e) < static_cast<unsigned>(none) ? e : none;
}

// Counts the rows of each adapter in a unit of consecutive rows: a warp to a unit, its counts in shared memory where they fit.
template <bool SHARED>
__global__ void __launch_bounds__(32) count_rows(const PlanParams p)
{
    extern __shared__ int counts_mem[];
    const int lane = threadIdx.x, groups = static_cast<int>(p.l.adapters) + 1;
    int* out = p.w + p.l.counts() + static_cast<int64_t>(blockIdx.x) * groups;
    volatile int* counts = SHARED ? counts_mem : out;
    ptx::grid_dependency_wait();
    for (int e = lane; e < groups; e += 32) counts[e] = 0;
    __syncwarp();
    const int64_t r0 = blockIdx.x * p.l.unit_rows, r1 = r0 + p.l.unit_rows < p.l.rows ? r0 + p.l.unit_rows : p.l.rows;
    for (int64_t r = r0 + lane; r - lane < r1; r += 32) {
        const int e = r < r1 ? adapter_of(p, r) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && (same & ((1u << lane) - 1u)) == 0u) counts[e] = counts[e] + __popc(same);
        __syncwarp();
    }
    if constexpr (SHARED)
        for (int e = lane; e < groups; e += 32) out[e] = counts[e];
    ptx::grid_launch_dependents();
}

constexpr int SCAN_THREADS = 1024;

// Exclusive sums of three values over the block's threads, and their totals.
__device__ __forceinline__ void block_scan(int (&v)[3], int (&total)[3], int (*warp_sums)[3])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int up = __shfl_up_sync(0xffffffffu, inc[i], o);
            if (lane >= o) inc[i] += up;
        }
    if (lane == 31)
        for (int i = 0; i < 3; ++i) warp_sums[warp][i] = inc[i];
    __syncthreads();
    int base[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        int s = warp_sums[lane][i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        total[i] = __shfl_sync(0xffffffffu, s, 31);
        base[i] = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
        if (warp == 0) base[i] = 0;
        v[i] = base[i] + inc[i] - v[i];
    }
    __syncthreads();
}

// One block: where each adapter's rows and pieces begin, and each unit's first position of every adapter.
__global__ void __launch_bounds__(SCAN_THREADS) scan_counts(const PlanParams p)
{
    __shared__ int warp_sums[32][3];
    const int groups = static_cast<int>(p.l.adapters) + 1;
    int* counts = p.w + p.l.counts();
    int *tiles = p.w + p.l.tile_starts(), *small = tiles + groups + 1;
    int carry[3] = {0, 0, 0};
    ptx::grid_dependency_wait();
    for (int e0 = 0; e0 < groups; e0 += SCAN_THREADS) {
        const int e = e0 + threadIdx.x;
        int n = 0;
        if (e < groups)
#pragma unroll 8
            for (int u = 0; u < static_cast<int>(p.l.units); ++u) n += counts[static_cast<int64_t>(u) * groups + e];
        int v[3] = {n, (n + TILE - 1) / TILE, (n + SMALL - 1) / SMALL}, total[3];
        block_scan(v, total, warp_sums);
        if (e < groups) {
            int at = carry[0] + v[0];
            p.w[e] = at;
            tiles[e] = carry[1] + v[1];
            small[e] = carry[2] + v[2];
#pragma unroll 8
            for (int u = 0; u < static_cast<int>(p.l.units); ++u) {
                int* c = counts + static_cast<int64_t>(u) * groups + e;
                const int m = *c;
                *c = at;
                at += m;
            }
        }
        for (int i = 0; i < 3; ++i) carry[i] += total[i];
    }
    if (threadIdx.x == 0) {
        p.w[groups] = carry[0];
        tiles[groups] = carry[1];
        small[groups] = carry[2];
    }
    ptx::grid_launch_dependents();
}

// The piece of number i, by the adapters' first numbers.
__device__ __forceinline__ Piece piece_of(const int* firsts, const int* starts, int groups, int i, int size)
{
    int lo = 0, hi = groups;  // firsts[lo] <= i < firsts[hi]
    if (i >= firsts[groups]) return Piece{0, 0, 0, 0};
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (firsts[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int first = starts[lo] + (i - firsts[lo]) * size, left = starts[lo + 1] - first;
    return Piece{lo, first, left < size ? left : size, 0};
}

// Warps of the first blocks put their unit's rows in order; the others write the tables.
template <bool SHARED>
__global__ void __launch_bounds__(32) place_rows(const PlanParams p)
{
    extern __shared__ int counts_mem[];
    const int lane = threadIdx.x, groups = static_cast<int>(p.l.adapters) + 1;
    ptx::grid_dependency_wait();
    const int64_t block = blockIdx.x;
    if (block >= p.l.units) {
        const int *tiles = p.w + p.l.tile_starts(), *small = tiles + groups + 1;
        Piece* out = reinterpret_cast<Piece*>(p.w + p.l.table());
        const int64_t i = (block - p.l.units) * 32 + lane;
        if (i < p.l.tiles)
            out[i] = piece_of(tiles, p.w, groups, static_cast<int>(i), TILE);
        else if (i < p.l.tiles + p.l.small)
            out[i] = piece_of(small, p.w, groups, static_cast<int>(i - p.l.tiles), SMALL);
        return;
    }
    int* from = p.w + p.l.counts() + block * groups;
    if constexpr (SHARED) {
        for (int e = lane; e < groups; e += 32) counts_mem[e] = from[e];
        __syncwarp();
    }
    volatile int* next = SHARED ? counts_mem : from;
    int* order = p.w + p.l.order();
    const int64_t r0 = block * p.l.unit_rows, r1 = r0 + p.l.unit_rows < p.l.rows ? r0 + p.l.unit_rows : p.l.rows;
    for (int64_t r = r0 + lane; r - lane < r1; r += 32) {
        const int e = r < r1 ? adapter_of(p, r) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int at = e >= 0 ? next[e] : 0;
        __syncwarp();
        if (e >= 0) {
            order[at + before] = static_cast<int>(r);
            if (before == 0) next[e] = at + __popc(same);
        }
        __syncwarp();
    }
}

bool plan_ok(int64_t rows, int64_t adapters) { return rows >= 0 && adapters >= 1 && rows <= MOST_ROWS && adapters <= MOST_ADAPTERS; }

}  // namespace ad
}  // namespace sgb

using namespace sgb;

extern "C" size_t adapter_plan_bytes(int64_t rows, int64_t adapters)
{
    return ad::plan_ok(rows, adapters) ? static_cast<size_t>(ad::PlanLayout(rows, adapters).words()) * 4 : 0;
}

extern "C" int adapter_plan(int64_t rows, int64_t adapters, const int32_t* index_dev, void* plan_dev, conv2d_stream_t stream)
{
    if (rows < 0 || adapters < 1) return CONV2D_ERR_INVALID;
    if (!ad::plan_ok(rows, adapters)) return CONV2D_ERR_UNSUPPORTED;
    if (!plan_dev || (rows > 0 && !index_dev)) return CONV2D_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(plan_dev) % 16 || reinterpret_cast<uintptr_t>(index_dev) % 4) return CONV2D_ERR_ALIGNMENT;
    const ad::PlanParams p{index_dev, static_cast<int*>(plan_dev), ad::PlanLayout(rows, adapters)};
    const int bytes = static_cast<int>((adapters + 1) * 4);
    const bool shared = bytes <= 40 * 1024;
    const int smem = shared ? bytes : 0;
    if (p.l.units > 0 && mx::launch(shared ? ad::count_rows<true> : ad::count_rows<false>, p.l.units, 32, smem, stream, 1, p) != cudaSuccess)
        return CONV2D_ERR_CUDA;
    if (mx::launch(ad::scan_counts, int64_t(1), ad::SCAN_THREADS, 0, stream, 1, p) != cudaSuccess) return CONV2D_ERR_CUDA;
    const int64_t tables = mx::cdiv<int64_t>(p.l.tiles + p.l.small, 32);
    if (p.l.units + tables > 0 &&
        mx::launch(shared ? ad::place_rows<true> : ad::place_rows<false>, p.l.units + tables, 32, smem, stream, 1, p) != cudaSuccess)
        return CONV2D_ERR_CUDA;
    return CONV2D_OK;
}
