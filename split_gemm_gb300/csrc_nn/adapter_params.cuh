// Kernel parameters of the adapter kernels and their shared memory.
#pragma once

#include <atomic>

#include "adapter_plan.cuh"

namespace sgb {
namespace ad {

constexpr int MOST_RANK = 128;

// How long a wait may take.  Tests compile the kernels with another time and with barriers that count an arrival which does not come: that of
// the first stage's rows, or of a product's end.  (As parameters of the kernels these cost 2% of a pass.)
#ifndef SGB_ADAPTER_WAIT_NS
#define SGB_ADAPTER_WAIT_NS 1000000000
#define SGB_ADAPTER_LOST_ROWS 0
#define SGB_ADAPTER_LOST_DONE 0
#endif
constexpr uint64_t WAIT_NS = SGB_ADAPTER_WAIT_NS;
constexpr int LOST_ROWS = SGB_ADAPTER_LOST_ROWS, LOST_DONE = SGB_ADAPTER_LOST_DONE;
constexpr uint64_t LAST_WAIT_NS = 1000000000;  // for what a CTA that is done with has in flight

struct PassParams {
    Plan plan;
    const __nv_bfloat16 *in, *w1, *w2;
    const float* scale;
    const void* base;  // y or dx0
    void* out;
    float* mid;
    uint32_t* status;
    int64_t in_stride, base_stride, out_stride;
    int adapters, rank, from, to;
    int relu;
    int splits;  // CTAs of a cluster
    int early;   // the next kernel may start: it waits itself for what it needs of this one
};

constexpr int P_BLOCK = P_STEP / 2;  // of `from`: in a block of operands
constexpr int P_MOST_STAGES = 4, P_MOST_CHUNKS = 8;
constexpr int P_ROOM = 227 * 1024;  // bytes of shared memory

// Bytes between the 16-byte columns of an MN-major block of w1: 16 more than they need, so that neighbours fall into different banks.
constexpr int W1_COLUMN = P_BLOCK * 16 + 16;

// Threads that finish chunks, and turns of base (64 bytes of each of them) on their way to shared memory.
constexpr int P_WARPS = 16, P_LOADERS = 32 * P_WARPS, P_DEPTH = 3;

// Shared memory by the rank padded to 16: an area that holds the first product's ring and, when that is over, the sums (from its start) and mid
// (to its end); when mid is in tensor memory, base's ring (to its end).  Before that lie w2's chunks, over the sums once those are joined; beside
// the area w2's first chunk, barriers and lists.  A chunk of w2: core matrices 144 bytes apart along the columns, so that the pairs that the
// backward pass places one by one fall into different banks, and 16 bytes more from one column of 8 ranks to the next, for the forward pass's vectors.
struct PassSmem {
    int rp;
    __host__ __device__ constexpr explicit PassSmem(int rank) : rp((rank + 15) / 16 * 16) {}
    // Accumulators of the first product, taken in turn: matrix units cut their sums off at fp32's last bit, towards zero, and a chain of 256 such
    // sums is off by 2.3e-6; eight chains of 32, joined by additions that round, by 2.8e-7 (fp32 throughout: 7e-7).
    __host__ __device__ constexpr int accumulators() const { return 512 / rp < 8 ? 512 / rp : 8; }
    __host__ __device__ constexpr int block() const { return TILE * P_BLOCK * 2 + (rp / 8 * W1_COLUMN + 1023) / 1024 * 1024; }
    __host__ __device__ constexpr int stage() const { return 2 * block(); }
    __host__ __device__ constexpr int column() const { return P_COLS / 8 * 144 + 16; }  // of a chunk: 8 ranks
    __host__ __device__ constexpr int chunk() const { return (rp / 8 * column() + 127) / 128 * 128; }
    __host__ __device__ constexpr int rest() const { return 512 + TILE * 4; }
    __host__ __device__ constexpr int area() const { return (P_ROOM - chunk() - rest()) / 128 * 128; }
    __host__ __device__ constexpr int stages() const { return area() / stage() < P_MOST_STAGES ? area() / stage() : P_MOST_STAGES; }
    __host__ __device__ constexpr int pitch() const { return rp + 4; }  // of the rows of sums and mid, in words
    __host__ __device__ constexpr int sums() const { return TILE * pitch() * 4; }  // and mid's bytes
    __host__ __device__ constexpr int ring() const { return P_DEPTH * P_LOADERS * 64; }
    __host__ __device__ constexpr int chunks() const { return 1 + (area() - ring()) / chunk() < P_MOST_CHUNKS ? 1 + (area() - ring()) / chunk() : P_MOST_CHUNKS; }
    // Those that lie neither over the sums nor over mid, if there are two; else all, to be filled when mid is in tensor memory.
    __host__ __device__ constexpr int apart() const { return 1 + (area() - ring() > sums() ? (area() - ring() - sums()) / chunk() : 0); }
    __host__ __device__ constexpr bool late() const { return apart() < 2; }
    __host__ __device__ constexpr int buffers() const { return late() || apart() > chunks() ? chunks() : apart(); }
};
static_assert(PassSmem(128).area() >= 2 * PassSmem(128).sums() && PassSmem(128).chunks() >= 2 && PassSmem(128).stages() >= 2 && PassSmem(128).ring() >= PassSmem(128).sums(),
              "the widest rank fits");

// Sums over the adapters' rows: out[e] (r, c) = sum of mid[t][r] * in[t][c].
struct SumJob {
    const __nv_bfloat16* in;
    const uint8_t *data, *scales;  // or a checkpoint
    const float* mid;
    float *out, *part;             // part: [2 * pieces][rank * cols], in out's order
    int64_t in_stride, blocks;     // blocks of 32 to a checkpoint's row
    int cols, col_blocks;
    int tiles_each;                // of a piece
    int mode;                      // 0: bf16 rows of whole vectors, 1: bf16, 2: a checkpoint
    int out_col;                   // 1: out[r][c]; else out[c][r]
    int mid_vec, out_vec, join_vec;
};

struct SumParams {
    Plan plan;
    SumJob jobs[2];  // without a result: not wanted
    uint32_t* status;
    int adapters, rank;
    int first_late;  // the first CTA of jobs[0], whose mid comes from the pass before
    int beside;      // that pass lets this kernel start early
};

int64_t sum_pieces(const PlanLayout& l, int tiles_each);
int launch_sums(SumParams& p, const PlanLayout& l, cudaStream_t stream);

// halved: tiles of 64 rows, not 128.
int launch_pass_fwd(const PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, bool halved, cudaStream_t stream);
// Up to rank 64.
int launch_small_fwd(PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, cudaStream_t stream);
int launch_pass_bwd(const PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, bool halved, cudaStream_t stream);

}  // namespace ad
}  // namespace sgb
