// Where each adapter's rows are: the plan that adapter calls share (adapter.h).
//
// A plan is a block of 32-bit words:
//   starts [adapters + 2]   position in `order` of each adapter's first row; [adapters]: of the rows without one; then rows
//   order  [rows]           rows by adapter, in their own order within it; those without one last
//   tiles  [most][4]        {adapter (adapters: none), first position, rows, 0}: the positions cut into pieces of at most
//                           TILE rows of one adapter; entries past the last have no rows
//   small  [..][4]          the same in pieces of at most SMALL rows, where rows <= SMALL_ROWS
//   counts [units][adapters + 1]   scratch of its making
#pragma once

#include "adapter_cuts.h"
#include "mx_common.cuh"

namespace sgb {
namespace ad {

static_assert(CARD_SMS == mx::SMS);
constexpr int SMALL = 8;
constexpr int64_t SMALL_ROWS = 640;
constexpr int64_t MOST_ROWS = (int64_t(1) << 31) - (1 << 16), MOST_ADAPTERS = 65535;

struct Piece {
    int adapter, first, rows, none;
};

struct PlanLayout {
    int64_t rows, adapters, tiles, small, units, unit_rows;
    __host__ __device__ PlanLayout(int64_t rows, int64_t adapters) : rows(rows), adapters(adapters)
    {
        const int64_t groups = adapters + 1 < rows ? adapters + 1 : rows;
        tiles = rows / TILE + groups;
        small = rows <= SMALL_ROWS ? rows / SMALL + groups : 0;
        // units of at least 256 rows, as many as a scratch of 2^22 words allows
        int64_t u = (rows + 255) / 256, most = (int64_t(1) << 22) / (adapters + 1);
        if (most > 1024) most = 1024;
        if (u > most) u = most;
        if (u < 1) u = 1;
        unit_rows = ((rows + u - 1) / u + 31) / 32 * 32;
        if (unit_rows < 32) unit_rows = 32;
        units = (rows + unit_rows - 1) / unit_rows;
    }
    // word offsets; the tables begin at 16 bytes
    __host__ __device__ int64_t order() const { return adapters + 2; }
    __host__ __device__ int64_t table() const { return (order() + rows + 3) / 4 * 4; }
    __host__ __device__ int64_t small_table() const { return table() + 4 * tiles; }
    __host__ __device__ int64_t tile_starts() const { return small_table() + 4 * small; }  // [2][adapters + 2]: pieces before each adapter's
    __host__ __device__ int64_t counts() const { return tile_starts() + 2 * (adapters + 2); }
    __host__ __device__ int64_t words() const { return counts() + units * (adapters + 1); }
};

// What kernels read of a plan.
struct Plan {
    const int *starts, *order;
    const Piece *tiles, *small;
    const int* tile_starts;  // [adapters + 2]: number of each adapter's first tile
    int n_tiles, n_small;
};

inline Plan plan_of(const void* plan, int64_t rows, int64_t adapters)
{
    const PlanLayout l(rows, adapters);
    const int* w = static_cast<const int*>(plan);
    return Plan{w, w + l.order(), reinterpret_cast<const Piece*>(w + l.table()), reinterpret_cast<const Piece*>(w + l.small_table()),
                w + l.tile_starts(), static_cast<int>(l.tiles), static_cast<int>(l.small)};
}

}  // namespace ad
}  // namespace sgb
